"""Device-side buffers and calls for the QSA path through the C ABI.

QSAPrefill / QSADecode own the caller-side device memory that the library
expects (caches, indexer state, outputs, workspace) as torch CUDA tensors and
call ``qsa_forward``. All arithmetic runs in libqsa.so.
"""
from __future__ import annotations

from typing import Dict

import torch

from . import qsa


def to_device(inp: Dict[str, torch.Tensor], device="cuda") -> Dict[str, torch.Tensor]:
    return {k: v.to(device, non_blocking=True).contiguous() for k, v in inp.items()}


GUARD_BYTES = 4096          # guard band on each side of a guarded output buffer
GUARD_WORD = 0x5A5A5A5A      # the pattern the bands are filled with, as int32 words


class Guarded:
    """A contiguous output tensor with a guard band of GUARD_BYTES on each side, filled
    with GUARD_WORD. `view` is the tensor handed to the library (256-byte aligned);
    intact() tells whether a call wrote outside it."""

    def __init__(self, shape, dtype, device="cuda"):
        n = 1
        for x in shape:
            n *= int(x)
        esz = torch.empty((), dtype=dtype).element_size()
        body = (n * esz + 255) // 256 * 256
        self.raw = torch.empty(2 * GUARD_BYTES + body, dtype=torch.uint8, device=device)
        self.raw.view(torch.int32).fill_(GUARD_WORD)
        self.body = body
        self.view = self.raw[GUARD_BYTES:GUARD_BYTES + n * esz].view(dtype).view(*shape)

    def intact(self) -> bool:
        lo = self.raw[:GUARD_BYTES].view(torch.int32)
        hi = self.raw[GUARD_BYTES + self.body:].view(torch.int32)
        want = GUARD_WORD
        return bool((lo == want).all().item()) and bool((hi == want).all().item())


def _outputs(shape_out, dtype, shape_sel, device, guard: bool):
    if not guard:
        return (torch.empty(shape_out, dtype=dtype, device=device),
                torch.empty(shape_sel, dtype=torch.int32, device=device), [])
    go, gs = Guarded(shape_out, dtype, device), Guarded(shape_sel, torch.int32, device)
    return go.view, gs.view, [go, gs]


class QSAPrefill:
    """One prefill call: compress every complete block, score, select, attend."""

    def __init__(self, w, inp: Dict[str, torch.Tensor], device="cuda", guard: bool = False):
        self.cfg = qsa.config_for(w)
        self.k = qsa.qsa_topk_blocks(self.cfg)
        g = to_device(inp, device)
        B, n_q = g["q"].shape[0], g["q"].shape[1]
        kv_cap = g["k"].shape[2]
        out, sel, self.guards = _outputs(g["q"].shape, g["q"].dtype, (B, n_q, self.k), device, guard)
        self.t = dict(q=g["q"], qi=g["qi"], k_cache=g["k"], v_cache=g["v"], ki_cache=g["ki"],
                      kbar_cache=torch.zeros(B, kv_cap // w.block, w.di, dtype=torch.float32, device=device),
                      kbar_blocks=torch.zeros(B, dtype=torch.int32, device=device),
                      kv_start=g["kv_start"], kv_len=g["kv_len"], q_first=g["q_first"], sel=sel, out=out)
        self.ws = qsa.alloc_workspace(self.cfg, qsa.QSA_PREFILL, B, n_q, kv_cap, device)

    def guards_intact(self) -> bool:
        """With guard=True: no call wrote past either end of `out` or `sel`."""
        return all(x.intact() for x in self.guards)

    def __call__(self, stream=None):
        qsa.qsa_forward(self.cfg, qsa.QSA_PREFILL, self.t, self.ws, stream)
        return self.t["out"], self.t["sel"]

    def status(self) -> int:
        return qsa.qsa_read_device_status(self.ws)


class QSADecode:
    """One decode step per sequence against caches holding kv_len - 1 tokens.

    The indexer state (k̄ for the complete blocks already in the cache) is built
    once by qsa_compress_blocks; each call appends the new token and runs the path.
    Calling again with the same kv_len re-appends the same token (the benchmark's
    steady-state step) -- reset_state() rewinds kbar_blocks for that.
    """

    def __init__(self, w, inp: Dict[str, torch.Tensor], device="cuda", guard: bool = False):
        self.cfg = qsa.config_for(w)
        self.k = qsa.qsa_topk_blocks(self.cfg)
        self.w = w
        g = to_device(inp, device)
        B = g["q"].shape[0]
        kv_cap = g["k"].shape[2]
        out, sel, self.guards = _outputs(g["q"].shape, g["q"].dtype, (B, 1, self.k), device, guard)
        self.t = dict(q=g["q"], qi=g["qi"], k_cache=g["k"], v_cache=g["v"], ki_cache=g["ki"],
                      kbar_cache=torch.zeros(B, kv_cap // w.block, w.di, dtype=torch.float32, device=device),
                      kbar_blocks=torch.zeros(B, dtype=torch.int32, device=device),
                      k_new=g["k_new"], v_new=g["v_new"], ki_new=g["ki_new"],
                      kv_start=g["kv_start"], kv_len=g["kv_len"], sel=sel, out=out)
        self.prev_len = (g["kv_len"] - 1).contiguous()
        # indexer state for the tokens already cached: k̄ of blocks [0, (L-1)/B) and
        # their count, both written by the library
        qsa.qsa_compress_blocks(self.cfg, self.t["ki_cache"], self.t["kv_start"], self.prev_len,
                                self.t["kbar_cache"], kbar_blocks=self.t["kbar_blocks"])
        self._blocks0 = self.t["kbar_blocks"].clone()
        self.ws = qsa.alloc_workspace(self.cfg, qsa.QSA_DECODE, B, 1, kv_cap, device)

    def reset_state(self):
        """Rewind the indexer state's block count to what it was before the first step."""
        self.t["kbar_blocks"].copy_(self._blocks0)

    def __call__(self, stream=None):
        qsa.qsa_forward(self.cfg, qsa.QSA_DECODE, self.t, self.ws, stream)
        return self.t["out"], self.t["sel"]

    def status(self) -> int:
        return qsa.qsa_read_device_status(self.ws)

    def guards_intact(self) -> bool:
        """With guard=True: no call wrote past either end of `out` or `sel`."""
        return all(x.intact() for x in self.guards)


class QSADecodeOffload(QSADecode):
    """QSADecode with the attention K/V cache in page-locked host memory: each call
    appends the new token to the host cache, selects on the device and copies only
    the attended blocks to the device staging buffer (qsa_decode_offload)."""

    def __init__(self, w, inp: Dict[str, torch.Tensor], device="cuda"):
        super().__init__(w, inp, device)
        self.t["k_cache"] = self.t["k_cache"].cpu().pin_memory()
        self.t["v_cache"] = self.t["v_cache"].cpu().pin_memory()
        self.staging = qsa.alloc_offload_staging(self.cfg, self.t["q"].shape[0], device)

    def __call__(self, stream=None):
        qsa.qsa_decode_offload(self.cfg, self.t, self.staging, self.ws, stream)
        return self.t["out"], self.t["sel"]


class QSAPaged:
    """A paged K/V cache and the steps that serve from it: chunks of prompts, drafted tokens, decode.

    Owns the pools [n_pages][Hkv][page_size][d], the page table and the indexer state (one plane per
    slot) of a fixed number of sequence slots, and the free pages. A step takes the packed rows of every
    slot's new tokens (a slot may have none), appends them with norm and rotation on the way and
    attends: over everything, or, given indexer rows, over the blocks that the indexer selects. Page
    numbers are handed out on the host; all arithmetic runs in libqsa.so.
    """

    def __init__(self, cfg, slots: int, max_len: int, n_pages: int, page_size: int, norm_rope=None, device="cuda"):
        B, di = cfg.indexer_compress_ratio, cfg.indexer_head_dim
        dt = torch.bfloat16 if cfg.dtype == qsa.QSA_DTYPE_BF16 else torch.float32
        self.cfg, self.nr, self.device, self.dtype = cfg, norm_rope, device, dt
        self.slots, self.max_len, self.page_size, self.n_pages = slots, max_len, page_size, n_pages
        pool = (n_pages, cfg.num_key_value_heads, page_size, cfg.head_dim)
        self.k_pages = torch.zeros(pool, dtype=dt, device=device)
        self.v_pages = torch.zeros(pool, dtype=dt, device=device)
        self.ki_cache = torch.zeros(slots, max_len, di, dtype=dt, device=device)
        self.kbar_cache = torch.zeros(slots, max_len // B, di, dtype=torch.float32, device=device)
        self.kbar_blocks = torch.zeros(slots, dtype=torch.int32, device=device)
        self.kv_start = torch.zeros(slots, dtype=torch.int32, device=device)
        self.table = torch.zeros(slots, -(-max_len // page_size), dtype=torch.int32)
        self.length = [0] * slots
        self.indexed = [0] * slots  # tokens with indexer keys
        self.pages = [[] for _ in range(slots)]
        self.free = list(range(n_pages - 1, -1, -1))
        self.ws = self.score_ws = None

    def release(self, slot: int):
        """The slot's sequence has ended: its pages go back."""
        self.free += reversed(self.pages[slot])
        self.pages[slot], self.length[slot], self.indexed[slot] = [], 0, 0
        self.kbar_blocks[slot] = 0

    def reserve(self, counts):
        """Room for counts[s] more tokens of every slot s: for all of them or, with an error, for none. The lengths
        count them from here on: the caller appends them itself (batch, qsa.qsa_paged_append). A step needs no
        call of this, it reserves its own."""
        self._take(counts, self._room(counts))

    def _room(self, counts):
        """Pages that counts[s] more tokens need in every slot s, or an error where there is no room."""
        if len(counts) != self.slots:
            raise ValueError(f"{len(counts)} counts for {self.slots} slots")
        need = []
        for s, n in enumerate(counts):
            if n < 0 or self.length[s] + n > self.max_len:
                raise ValueError(f"slot {s}: {self.length[s]} + {n} tokens, room for {self.max_len}")
            need.append(-(-(self.length[s] + n) // self.page_size) - len(self.pages[s]))
        if sum(need) > len(self.free):
            raise ValueError(f"{sum(need)} pages needed, {len(self.free)} free")
        return need

    def _take(self, counts, need):
        for s, (n, m) in enumerate(zip(counts, need)):
            for _ in range(m):
                self.table[s, len(self.pages[s])] = self.free[-1]
                self.pages[s].append(self.free.pop())
            self.length[s] += n

    def _give_back(self, counts, need):
        """_take undone, with the free pages in the order that they had."""
        for s in reversed(range(self.slots)):
            for _ in range(need[s]):
                self.free.append(self.pages[s].pop())
            self.length[s] -= counts[s]

    def batch(self, counts):
        """The packed batch of counts[s] new tokens of every slot, whose lengths count them already."""
        start = torch.tensor([0] + list(counts)).cumsum(0).to(torch.int32)
        lens = torch.tensor(self.length, dtype=torch.int32)
        return qsa.make_paged(start.to(self.device), lens.to(self.device), self.table.to(self.device),
                              n_tok=sum(counts), max_chunk=max(counts), page_size=self.page_size, n_pages=self.n_pages)

    def select(self, counts, qi, pg):
        """Selection [n_tok][k] of the packed rows qi [n_tok][Hi][di]: compresses the blocks that the step
        completed, then scores and selects with every slot's rows padded to the longest chunk (slots * max(counts)
        rows of indexer queries and lists, whatever n_tok is)."""
        cfg, most = self.cfg, max(counts)
        done = self.kbar_blocks.clone()  # a tensor of its own: a step that is refused later takes the old one back
        qsa.qsa_compress_blocks(cfg, self.ki_cache, self.kv_start, pg.kv_len, self.kbar_cache,
                                blocks_done=self.kbar_blocks, kbar_blocks=done)
        self.kbar_blocks = done
        count = torch.tensor(counts)
        seq = torch.repeat_interleave(torch.arange(self.slots), count).to(self.device)
        row = torch.cat([torch.arange(c) for c in counts]).to(self.device)
        padded = torch.zeros(self.slots, most, *qi.shape[1:], dtype=self.dtype, device=self.device)
        padded[seq, row] = qi
        sel = torch.empty(self.slots, most, qsa.qsa_topk_blocks(cfg), dtype=torch.int32, device=self.device)
        self.score_ws = self._grown(self.score_ws, qsa.qsa_workspace_size(cfg, qsa.QSA_PREFILL, self.slots, most, self.max_len))
        q_first = pg.kv_len - count.to(torch.int32).to(self.device)
        qsa.qsa_index_score_topk(cfg, padded, self.kbar_cache, pg.kv_len, q_first, self.max_len, sel, self.score_ws)
        return sel[seq, row].contiguous()

    def step(self, counts, q, k, v, qi=None, ki=None):
        """counts[s] new tokens of every slot s, packed in that order: q [n_tok][Hq][d] and k, v
        [n_tok][Hkv][d] before norm and rotation. With the indexer's qi [n_tok][Hi][di] (rotated) and ki
        [n_tok][di] the step attends the selected blocks; a slot whose earlier tokens came without them
        cannot. Returns [n_tok][Hq][d]. A step that raises leaves the slots as they were. It copies geometry and
        page table from the host, so it cannot be captured into a graph; the calls that it makes can."""
        need = self._room(counts)
        cfg, n = self.cfg, sum(counts)
        heads, kv = (n, cfg.num_attention_heads, cfg.head_dim), (n, cfg.num_key_value_heads, cfg.head_dim)
        want = [("q", q, heads), ("k", k, kv), ("v", v, kv)]
        if (qi is None) != (ki is None):
            raise ValueError("qi and ki come together")
        if ki is not None:
            want += [("qi", qi, (n, cfg.indexer_n_heads, cfg.indexer_head_dim)), ("ki", ki, (n, cfg.indexer_head_dim))]
            for s, c in enumerate(counts):
                if c and self.indexed[s] != self.length[s]:
                    raise ValueError(f"slot {s}: {self.length[s]} tokens, {self.indexed[s]} of them with indexer keys")
        for name, t, shape in want:
            if tuple(t.shape) != shape or t.dtype != self.dtype:
                raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype}, expected {shape} {self.dtype}")
        if n == 0:
            return torch.empty_like(q)
        # Any of the calls below may still refuse (strides, alignment, devices, norm weights, sizes that no
        # kernel serves): the slots are then as they were. What the calls before it wrote lies behind the slots'
        # tokens, where the next step writes again.
        blocks = self.kbar_blocks
        self._take(counts, need)
        try:
            pg = self.batch(counts)
            self.ws = self._grown(self.ws, qsa.qsa_paged_workspace_size(cfg, pg))
            turned, out = torch.empty_like(q), torch.empty_like(q)
            qsa.qsa_paged_append(cfg, self.nr, pg, k, v, self.k_pages, self.v_pages, self.ws, q=q, q_out=turned, ki=ki,
                                 ki_cache=self.ki_cache if ki is not None else None)
            sel = self.select(counts, qi, pg) if ki is not None else None
            qsa.qsa_paged_attn(cfg, pg, turned, self.k_pages, self.v_pages, sel, out, self.ws)
        except BaseException:
            self._give_back(counts, need)
            self.kbar_blocks = blocks
            raise
        if ki is not None:
            self.indexed = [a + c for a, c in zip(self.indexed, counts)]
        return out

    def _grown(self, ws, need: int):
        """ws, or a larger one that keeps its status word."""
        if ws is not None and ws.numel() >= need:
            return ws
        new = torch.zeros(need, dtype=torch.uint8, device=self.device)
        if ws is not None:
            new[:256] = ws[:256]
        return new

    def status(self) -> int:
        """First device status of the steps since the last reading (QSA_OK before the first step)."""
        codes = [qsa.qsa_read_device_status(ws) for ws in (self.ws, self.score_ws) if ws is not None]
        return next((c for c in codes if c != qsa.QSA_OK), qsa.QSA_OK)
