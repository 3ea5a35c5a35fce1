"""The synthetic decode layer, composed from the library's C ABI.

One layer of the layer-stack workload (attention core excluded):
  [q | kv] = x·[Wq; Wkv]ᵀ          one fused projection (dec_linear)
  r        = bf16(x + q·Woᵀ)        o projection reading q in place from the
                                    fused output, residual fused (dec_linear_ex)
  x'       = bf16(r + MoE(r))       the MoE decode block with its shared expert
                                    and the residual fused (moe_decode_residual)
and, on a side stream, an L2 prefetch of the next layer's weights. The o
projection consuming q stands in for the attention output; kv is computed and
not consumed. The benchmark and the full-size parity tests both run this
function, so what is timed is what is checked. attention_layer is the same
layer with its attention over a paged cache, w4_layer that one with its norms
and with 4-bit weights in its projections.

Sources: "vLLM 如何用智能体辅助优化 Kimi K3 解码性能", Part 1 §1 (projections),
§3 (MoE block, shared expert on its own stream) and §4 (prefetch of upcoming
weights on a side stream); "vLLM 宣布 Kimi K3 在 GB300 NVL72 上实现 batch 1 解码
842 tokens/s", the per-layer kernel trace (a layer as the unit of work).
"""
from __future__ import annotations

from . import (dec_linear, dec_linear_w4, dec_rmsnorm, dec_rmsnorm_mx, kv_append, kv_attention,
               l2_prefetch, moe_decode)


def decode_layer(L, x, qkv, r, out, topk, idx=None, stream=None, prefetch=None):
    """Enqueue one decode layer on ``stream``; returns ``out``.

    L: weights with Wqkv [H+KV, H], Wo [H, H], Wr, W13, W2, Ws13, Ws2 (bf16,
    on the device). x [M, H] bf16 input; qkv [M, H+KV], r [M, H] and out
    [M, H] bf16 buffers the caller owns (out may alias x). idx: optional
    [M, topk] int32 for the chosen experts. prefetch: optional
    (side_stream, event, ptr, nbytes) -- the range is pulled into L2 on the
    side stream once the o projection has been enqueued.
    """
    H = x.shape[1]
    dec_linear(x, L.Wqkv, qkv, stream=stream)
    dec_linear(qkv[:, :H], L.Wo, r, stream=stream, residual=x)
    if prefetch is not None:
        side, ev, ptr, nbytes = prefetch
        ev.record(stream)
        side.wait_event(ev)
        l2_prefetch(ptr, nbytes, stream=side)
    moe_decode(r, L.Wr, L.W13, L.W2, L.Ws13, L.Ws2, topk, out=out, topk_idx=idx, stream=stream,
               residual=r)
    return out


def attention_layer(L, x, kv, rope, qkv, o, r, out, topk, wq=None, wk=None, window=0, idx=None,
                    stream=None, prefetch=None, interleaved=False):
    """One decode layer with its attention; returns ``out``.

      [q | k | v] = x·Wqkvᵀ          the fused projection (dec_linear)
      q, k        normed and rotated per head, k and v to the cache (kv_append,
                  the queries in place in qkv)
      o           = attention of the new tokens over the cache (kv_attention)
      r           = bf16(x + o·Woᵀ),  x' = bf16(r + MoE(r)) as decode_layer

    L: as decode_layer, Wqkv [q width + 2*kv.heads*kv.dim, H], Wo [H, q width].
    kv: PagedKV of this layer, whose kv_len already counts the step's tokens
    (kv_resize does that once for all layers); at most 64 tokens in all. rope,
    wq, wk, interleaved: see kv_append. qkv, r, out: buffers as decode_layer's;
    o [M, q width] bf16. The other arguments as there.
    """
    dec_linear(x, L.Wqkv, qkv, stream=stream)
    q = kv_append(qkv, kv, rope, wq, wk, q=qkv[:, :L.Wo.shape[1]], stream=stream,
                  interleaved=interleaved)
    kv_attention(q, kv, out=o, window=window, stream=stream)
    dec_linear(o, L.Wo, r, stream=stream, residual=x)
    if prefetch is not None:
        side, ev, ptr, nbytes = prefetch
        ev.record(stream)
        side.wait_event(ev)
        l2_prefetch(ptr, nbytes, stream=side)
    moe_decode(r, L.Wr, L.W13, L.W2, L.Ws13, L.Ws2, topk, out=out, topk_idx=idx, stream=stream,
               residual=r)
    return out


def w4_layer(L, x, kv, rope, qkv, o, a, r, out, topk, wq=None, wk=None, window=0, idx=None, stream=None,
             interleaved=False, mx=True, eps=1e-6):
    """One decode layer with its norms, attention and 4-bit projections; returns ``out``.

      n           = norm(x)·w1          in 8 bits with scales (dec_rmsnorm_mx), or with
                                        mx=False in bf16 (dec_rmsnorm)
      [q | k | v] = n·Wqkvᵀ             4-bit weights (dec_linear_w4)
      o           = attention, as attention_layer
      a           = o·Woᵀ               4-bit weights
      r           = bf16(x + a),  n = norm(r)·w2      (dec_rmsnorm, one pass)
      x'          = bf16(r + MoE(n))    (moe_decode, bf16 weights)

    L: weights with Wqkv [q width + 2*kv.heads*kv.dim, H] and Wo [H, q width] as W4
    (dec_quant_w4), w1 and w2 [H] bf16, Wr, W13, W2, Ws13, Ws2 as decode_layer's.
    x [M, H] bf16, M <= 64; qkv, o, r, out: buffers as attention_layer's, a [M, H]
    bf16. out may be x. The other arguments as there; H a multiple of 32 for mx.
    """
    norm = dec_rmsnorm_mx if mx else dec_rmsnorm
    dec_linear_w4(norm(x, L.w1, eps=eps, stream=stream), L.Wqkv, qkv, stream=stream)
    q = kv_append(qkv, kv, rope, wq, wk, q=qkv[:, :L.Wo.k], stream=stream, interleaved=interleaved)
    kv_attention(q, kv, out=o, window=window, stream=stream)
    dec_linear_w4(o, L.Wo, a, stream=stream)
    n, _ = dec_rmsnorm(a, L.w2, x, h=r, eps=eps, stream=stream)
    moe_decode(n, L.Wr, L.W13, L.W2, L.Ws13, L.Ws2, topk, out=out, topk_idx=idx, stream=stream,
               residual=r)
    return out
