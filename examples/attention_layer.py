"""One attention layer of a serving model, end to end in FP8 on one GPU.

The projections are block-scaled FP8 GEMMs, the keys and values go to a paged FP8 cache, and the
attention reads them there:

    x -> cast -> fp8_gemm_nt (q, k, v) -> fp8_kv_cache_write -> fp8_paged_attention -> cast -> fp8_gemm_nt

Two sequences of different length are fed as a chunk of their prompts, a second chunk, and then token by
token; the same tokens fed in one chunk have to give the same result.  At the end one sequence is moved
to a cache with other pages (fp8_kv_cache_read, fp8_kv_cache_write), which must not change its values.

    python examples/attention_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_amd as dg  # noqa: E402

DEV = torch.device("cuda", 0)
HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 1024, 16, 4, 64, 16


def quantise_weight(w):
    """FP32 [n, k] -> E4M3 codes and one scale per 128 x 128 block."""
    n, k = w.shape
    blocks = w.view(n // 128, 128, k // 128, 128)
    scale = blocks.abs().amax((1, 3)) / 448.0
    codes = (blocks / scale[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(n, k), scale.contiguous()


def linear(x, weight):
    """x [m, k] BF16 times weight.T, through the FP8 GEMM."""
    out = torch.empty((x.shape[0], weight[0].shape[0]), dtype=torch.bfloat16, device=x.device)
    return dg.fp8_gemm_nt(dg.per_token_group_cast_fp8(x), weight, out)


class AttentionLayer:
    def __init__(self, pages, sequences, seed=0, window=0, sinks=0):
        g = torch.Generator(DEV).manual_seed(seed)
        self.window, self.sinks = window, sinks
        self.w_qkv = quantise_weight(torch.randn(((HEADS + 2 * KV_HEADS) * DIM, HIDDEN), generator=g, device=DEV) * HIDDEN ** -0.5)
        self.w_out = quantise_weight(torch.randn((HIDDEN, HEADS * DIM), generator=g, device=DEV) * (HEADS * DIM) ** -0.5)
        self.k_cache, self.v_cache = dg.fp8_kv_cache_empty(pages, KV_HEADS, PAGE, DIM, device=DEV)
        # every sequence owns a run of pages, handed out in any order
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        self.table = order[: pages // sequences * sequences].view(sequences, -1).contiguous()
        self.lens = [0] * sequences

    def slots(self, seq, first, n):
        at = torch.arange(first, first + n, device=DEV)
        return self.table[seq, at // PAGE].long() * PAGE + at % PAGE

    def forward(self, x, new):
        """x [sum(new), HIDDEN] BF16: the next new[b] tokens of each sequence b, one after the other."""
        total = x.shape[0]
        qkv = linear(x, self.w_qkv).view(total, HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split((HEADS, KV_HEADS, KV_HEADS), dim=1)
        slots = torch.cat([self.slots(b, self.lens[b], n) for b, n in enumerate(new)])
        dg.fp8_kv_cache_write(k, v, self.k_cache, self.v_cache, slots)
        self.lens = [a + n for a, n in zip(self.lens, new)]
        cu = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
        out = dg.fp8_paged_attention(q, self.k_cache, self.v_cache, self.table, torch.tensor(self.lens, dtype=torch.int32, device=DEV),
                                     cu_seqlens_q=cu, max_seqlen_q=max(new), max_seqlen_k=max(self.lens), window=self.window,
                                     sinks=self.sinks)
        return linear(out.view(total, HEADS * DIM), self.w_out)


def main(window=0, sinks=0):
    lens = [300, 77]
    g = torch.Generator(DEV).manual_seed(1)
    x = [torch.randn((n, HIDDEN), generator=g, device=DEV).bfloat16() for n in lens]

    whole = AttentionLayer(64, 2, window=window, sinks=sinks)
    want = whole.forward(torch.cat(x), lens).split(lens)

    layer = AttentionLayer(64, 2, window=window, sinks=sinks)
    got = [[], []]
    at = [0, 0]
    for new in [[200, 40], [80, 30]] + [[1, 1]] * 7 + [[13, 0]]:
        y = layer.forward(torch.cat([x[b][at[b]: at[b] + n] for b, n in enumerate(new)]), new).split(new)
        for b, n in enumerate(new):
            got[b].append(y[b])
            at[b] += n
    assert at == lens
    # The same keys and values bit for bit, whatever the chunks; outputs up to the order of sums.
    for a, b in zip((*whole.k_cache, *whole.v_cache), (*layer.k_cache, *layer.v_cache)):
        assert torch.equal(a, b)
    off = max(float((torch.cat(got[b]).float() - want[b].float()).norm() / want[b].float().norm()) for b in range(2))
    print(f"chunks and single tokens against one chunk: relative difference {off:.2g}")

    # move sequence 0 to a cache with larger pages
    k, v = dg.fp8_kv_cache_read(layer.k_cache, layer.v_cache, layer.slots(0, 0, lens[0]))
    k2, v2 = dg.fp8_kv_cache_empty(5, KV_HEADS, 64, DIM, device=DEV)
    slots = torch.arange(lens[0], device=DEV)
    dg.fp8_kv_cache_write(k, v, k2, v2, slots)
    again = dg.fp8_kv_cache_read(k2, v2, slots)
    moved = torch.equal(k, again[0]) and torch.equal(v, again[1])
    print(f"moved to other pages: values {'unchanged' if moved else 'CHANGED'}")
    return off, moved


if __name__ == "__main__":
    off, moved = main()
    sys.exit(0 if off < 0.02 and moved else 1)
