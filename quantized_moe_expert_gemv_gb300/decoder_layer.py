"""A decoder layer on the library's calls, as a serving loop would make them: prompts enter an 8-bit cache, tokens
are decoded over it, and each kv head's cache goes back to a budget of its heaviest pages.

    python -m quantized_moe_expert_gemv_gb300.decoder_layer

Attention block: RMSNorm, the fused query/key/value projection, rotary positions (torch), then
si_kv_append, si_kv_attend, si_kv_weigh, the output projection and the residual.  FFN block: the pre-normed
quantised mixture of experts (si_moe_forward_prefill for prompts, si_moe_forward_decode for steps of up to four
sequences).  si_kv_evict runs whenever a sequence's full pages exceed the budget.  The weights are synthetic.
"""
from __future__ import annotations

import math

import torch

from . import binding as si
from . import device, synth


class DecoderLayer:
    """One layer and the caches of up to four sequences."""

    def __init__(self, shape: synth.MoeShape, heads: int, kv: int, dim: int, page: int = 64, code: str = "int8",
                 n_seqs: int = 4, max_len: int = 4096, budget: int = 32, sink: int = 1, recent: int = 4, window: int = 32,
                 decay: float = 0.98, seed: int = 1, dev: str = "cuda:0"):
        if not 1 <= n_seqs <= si.SI_MAX_DECODE_TOKENS:
            raise ValueError(f"1 to {si.SI_MAX_DECODE_TOKENS} sequences")
        si.load_library()
        self.shape, self.heads, self.kv, self.dim, self.page, self.dev = shape, heads, kv, dim, page, dev
        self.n, self.max_len, self.budget, self.sink, self.recent = n_seqs, max_len, budget, sink, recent
        self.window, self.decay, self.sm = window, decay, 1.0 / math.sqrt(dim)
        g = torch.Generator(device=dev).manual_seed(seed)
        hidden = shape.hidden

        def weight(*size):
            return (torch.randn(size, generator=g, device=dev) / math.sqrt(size[-1])).bfloat16()
        self.w_qkv, self.w_out = weight((heads + 2 * kv) * dim, hidden), weight(hidden, heads * dim)
        self.norm = torch.rand(hidden, generator=g, device=dev) + 0.5
        self.layer = device.to_device(synth.make_layer(shape, seed=seed), dev)
        self.layer.norm_weight, self.layer.norm_eps = synth_gain(shape, seed, dev), 1e-6
        self.moe = si.si_moe_plan(device.desc_for(shape, max_tokens=n_seqs * max_len), 0)
        self.moe_step = device.alloc_scratch(self.moe, si.SI_MODE_DECODE, n_seqs, dev)

        # the cache: pages for the sequences, and as many again as an eviction fills
        self.columns = max_len // page
        n_pages = n_seqs * (self.columns + budget)
        full = (n_pages, kv, page, dim)
        kind = torch.int8 if code == "int8" else torch.float8_e4m3fn
        self.plan = si.si_kv_plan(si.make_kv_desc(heads, kv, dim, page, code, "bf16"))
        self.tensors = [torch.zeros(full, dtype=kind, device=dev), torch.zeros(full, dtype=kind, device=dev),
                        torch.zeros(full[:2], device=dev), torch.zeros(full[:2], device=dev),
                        torch.zeros((n_seqs, kv, 2 * page, dim), dtype=torch.bfloat16, device=dev),
                        torch.zeros((n_seqs, kv, 2 * page, dim), dtype=torch.bfloat16, device=dev)]
        self.cache = si.kv_cache(*self.tensors)
        self.free = list(range(n_pages))
        self.pages = [[] for _ in range(n_seqs)]        # the sequences' pages, in order
        self.table = torch.full((n_seqs, self.columns), -1, dtype=torch.int32, device=dev)
        self.lens, self.lens_next = (torch.zeros(n_seqs, dtype=torch.int32, device=dev) for _ in range(2))
        self.host_lens = [0] * n_seqs                   # the same on the host, which hands out the pages
        self.positions = [0] * n_seqs                   # tokens seen, evicted ones among them
        self.acc, self.acc_next = (torch.zeros((n_seqs, kv, max_len), device=dev) for _ in range(2))
        # scratch for the largest call, once: the errors that the device reports lie in it until they are read
        need = si.si_kv_scratch_bytes(self.plan, n_seqs, n_seqs * max_len, max_len, max_len)
        self.scratch = torch.empty(need, dtype=torch.uint8, device=dev)
        si.si_kv_scratch_init(self.plan, self.scratch)

    # ---------------------------------------------------------------- pieces
    def _batch(self, counts, lens) -> si.si_kv_batch:
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        q_start = torch.tensor(starts, dtype=torch.int32, device=self.dev)
        return si.kv_batch(self.n, starts[-1], max(counts), self.max_len, q_start, lens, self.table)

    def _reserve(self, counts) -> None:
        """Pages for the ones that the new tokens complete."""
        for b, n in enumerate(counts):
            while len(self.pages[b]) < (self.host_lens[b] + n) // self.page:
                self.pages[b].append(self.free.pop())
                self.table[b, len(self.pages[b]) - 1] = self.pages[b][-1]

    def _rotate(self, x: torch.Tensor, pos: torch.Tensor) -> torch.Tensor:
        half = self.dim // 2
        angle = pos.double()[:, None] * torch.pow(10000.0, -torch.arange(half, device=self.dev).double() / half)
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
        a, b = x[..., :half].float(), x[..., half:].float()
        return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2).to(x.dtype)

    def attention(self, x: torch.Tensor, counts) -> torch.Tensor:
        """x [rows, hidden] bf16, counts[b] rows of sequence b: x + the attention block's output."""
        h, kv, d, rows = self.heads, self.kv, self.dim, x.shape[0]
        y = x.float()
        y = (y * torch.rsqrt(y.square().mean(1, keepdim=True) + 1e-6) * self.norm).bfloat16()
        qkv = torch.nn.functional.linear(y, self.w_qkv).view(rows, h + 2 * kv, d)
        pos = torch.cat([torch.arange(p, p + n, device=self.dev) for p, n in zip(self.positions, counts)])
        qk = self._rotate(qkv[:, :h + kv], pos)
        q, k, v = qk[:, :h], qk[:, h:], qkv[:, h + kv:]   # strided views: no copies

        self._reserve(counts)
        si.si_kv_append(self.plan, self.cache, self._batch(counts, self.lens), k, v, self.lens_next, self.scratch)
        self.lens, self.lens_next = self.lens_next, self.lens
        for b, n in enumerate(counts):
            self.host_lens[b] += n
            self.positions[b] += n
        out = torch.empty((rows, h, d), dtype=torch.bfloat16, device=self.dev)
        lse = torch.empty((rows, h), device=self.dev)
        si.si_kv_attend(self.plan, self.cache, self._batch(counts, self.lens), q, out, lse, self.sm, self.scratch)
        self._weigh(counts, q, lse)
        self.last = (q, out, lse)
        return x + torch.nn.functional.linear(out.view(rows, h * d), self.w_out)

    def _weigh(self, counts, q, lse) -> None:
        """The weights that each sequence's last rows (a window of a prompt, or the step's one) gave the cache."""
        last = [min(n, self.window) for n in counts]
        if last != list(counts):
            at, rows = 0, []
            for b, (n, m) in enumerate(zip(counts, last)):
                rows += range(at + n - m, at + n)
                at += n
                # new tokens before the window have no earlier sum: what lies in their place is an evicted one's
                self.acc[b, :, self.host_lens[b] - n:self.host_lens[b] - m] = 0
            rows = torch.tensor(rows, device=self.dev)
            q, lse = q[rows], lse[rows]
        si.si_kv_weigh(self.plan, self.cache, self._batch(last, self.lens), q, lse, self.acc, self.acc, self.decay, self.sm,
                       self.scratch)

    def evict(self) -> bool:
        """Back to the budget, where a sequence is past it: the kept pages move to fresh ones, the old ones are free."""
        if max(len(p) for p in self.pages) <= self.budget:
            return False
        fresh = [[self.free.pop() for _ in range(min(len(p), self.budget))] for p in self.pages]
        new_table = torch.tensor([p + [-1] * (self.budget - len(p)) for p in fresh], dtype=torch.int32, device=self.dev)
        keep = torch.empty((self.n, self.kv, self.budget), dtype=torch.int32, device=self.dev)
        si.si_kv_evict(self.plan, self.cache, self._batch([0] * self.n, self.lens), self.acc, self.acc_next, self.budget,
                       self.sink, self.recent, new_table, None, keep, self.lens_next, self.scratch)
        self.lens, self.lens_next = self.lens_next, self.lens
        self.acc, self.acc_next = self.acc_next, self.acc
        self.table.fill_(-1)
        self.table[:, :self.budget] = new_table
        for b, pages in enumerate(self.pages):
            self.free += pages
            self.host_lens[b] = len(fresh[b]) * self.page + self.host_lens[b] % self.page
        self.pages, self.kept = fresh, keep
        return True

    # ---------------------------------------------------------------- calls
    def prompts(self, x: torch.Tensor, counts) -> torch.Tensor:
        """x [rows, hidden] bf16, the sequences' prompts one after the other; the layer's output, bf16."""
        h = self.attention(x, counts).contiguous()
        out = torch.empty(h.shape, dtype=torch.float32, device=self.dev)
        scratch = device.alloc_scratch(self.moe, si.SI_MODE_PREFILL, h.shape[0], self.dev)
        si.si_moe_forward_prefill(self.moe, self.layer.struct(), h, h.shape[0], out, None, scratch)
        if si.si_moe_read_status(self.moe, scratch) != si.SI_OK:
            raise RuntimeError("the expert block reported an error")
        self.evict()
        return out.bfloat16()

    def step(self, x: torch.Tensor) -> torch.Tensor:
        """x [n_seqs, hidden] bf16, one token of each sequence; the layer's output, bf16."""
        h = self.attention(x, [1] * self.n).contiguous()
        out = torch.empty(h.shape, dtype=torch.float32, device=self.dev)
        si.si_moe_forward_decode(self.moe, self.layer.struct(), h, self.n, out, None, self.moe_step)
        self.evict()
        return out.bfloat16()

    def status(self) -> int:
        """The first error that a call of either block recorded on the device (SI_OK if none)."""
        st = si.si_kv_read_status(self.plan, self.scratch)
        return st if st != si.SI_OK else si.si_moe_read_status(self.moe, self.moe_step)


def synth_gain(shape: synth.MoeShape, seed: int, dev: str) -> torch.Tensor:
    return torch.from_numpy(synth.make_norm_weight(shape, seed)).to(dev)


def main() -> None:
    torch.cuda.set_device(0)
    layer = DecoderLayer(synth.QWEN3_30B_A3B, heads=32, kv=4, dim=128, budget=16)
    counts = [700, 1500, 64, 1023]
    g = torch.Generator(device="cuda:0").manual_seed(7)
    x = torch.randn((sum(counts), layer.shape.hidden), generator=g, device="cuda:0").bfloat16()
    y = layer.prompts(x, counts)
    print(f"prompts of {counts} tokens; cache lengths now {layer.lens.tolist()}")
    ends = torch.tensor(counts, device="cuda:0").cumsum(0) - 1
    x, begin, end = y[ends], torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    steps = 200
    for i in range(steps):
        if i == 20:
            begin.record()
        x = layer.step(x)
        x = x / x.float().square().mean(1, keepdim=True).sqrt().clamp(min=1e-3).to(x.dtype)  # (a layer's output stands for its input)
    end.record()
    torch.cuda.synchronize()
    if layer.status() != si.SI_OK:
        raise RuntimeError(si.si_status_string(layer.status()))
    print(f"{steps} steps of {layer.n} tokens, {begin.elapsed_time(end) / (steps - 20) * 1e3:.0f} us each; "
          f"cache lengths {layer.lens.tolist()} of {layer.positions} tokens seen, budget {layer.budget} pages of {layer.page}")


if __name__ == "__main__":
    main()
