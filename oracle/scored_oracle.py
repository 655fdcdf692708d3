"""fp64 statement of attention with capped, biased or range-masked scores (test
infrastructure only).

For the query row at position p and q head h, with x_j = scale * q . k_j:
    score_j = cap(x_j) - slope_h * |p - j|,   cap(x) = softcap * tanh(x / softcap) or x,
softmax over the keys begin <= j < end of the row; a row without keys is 0.
Masked keys are left out before any arithmetic, so what they hold (NaN,
infinity) cannot reach the result. The pages name no such scores: the formulas
are the definition.
"""

from __future__ import annotations

import numpy as np

from .paged_oracle import bf16_bits_to_f64


def scored_attention(q, kv_cache, block_table, seq_lens, query_start_loc, num_computed, scale,
                     softcap=0.0, slopes=None, key_begin=None, key_end=None):
    """(out, bound) fp64 [T, Hq, D] of one step whose new tokens are in the
    cache. `bound` is how far an fp32 kernel with bf16 softmax weights and a
    bf16 output may be from `out`. With w the softmax weights and A = sum w|v|:
      - a weight rounded to bf16 is off by 2^-8 of itself:  2^-8 A;
      - the output rounded to bf16 is off by 2^-8 |out|;
      - a score off by at most e moves every weight by a factor within
        e^(+-e), and the normalisation by another: 2 e A. e: the fp32 sum of
        D products, D 2^-24 scale sum |q||k|, and 16 roundings of the score
        and of the bias (scaling, cap, bias, base change, exponential, online
        rescaling), 16 * 2^-24 (|score| + |bias| + 1);
      - l and o summed in fp32 over n keys: 2 n 2^-24 A.
    A tenth is added for the products of these."""
    B, Hkv = kv_cache.shape[2], kv_cache.shape[3]
    T, Hq, D = q.shape
    G = Hq // Hkv
    out = np.zeros((T, Hq, D))
    bound = np.zeros((T, Hq, D))
    qf = bf16_bits_to_f64(q)
    for r in range(len(seq_lens)):
        t0, t1, c, L = (int(query_start_loc[r]), int(query_start_loc[r + 1]), int(num_computed[r]),
                        int(seq_lens[r]))
        for t in range(t0, t1):
            p = c + t - t0
            lo = 0 if key_begin is None else max(0, int(key_begin[t]))
            hi = p + 1 if key_end is None else min(L, int(key_end[t]))
            if lo >= hi:
                continue
            j = np.arange(lo, hi)
            blk = block_table[r][j // B].astype(np.int64)
            assert (blk >= 0).all()
            K = bf16_bits_to_f64(kv_cache[blk, 0, j % B])  # [n, Hkv, D]
            V = bf16_bits_to_f64(kv_cache[blk, 1, j % B])
            qr = qf[t].reshape(Hkv, G, D)
            x = scale * np.einsum("hgd,nhd->hgn", qr, K)
            mass = scale * np.einsum("hgd,nhd->hgn", np.abs(qr), np.abs(K)).max(axis=2)
            if softcap:
                x = softcap * np.tanh(x / softcap)
            size = np.abs(x).max(axis=2)
            if slopes is not None:
                bias = slopes.astype(np.float64).reshape(Hkv, G, 1) * np.abs(p - j)
                near = np.abs(slopes.astype(np.float64)).reshape(Hkv, G) * \
                    (np.abs(p - j).max() - np.abs(p - j).min())
                x = x - bias
                size = size + near
            w = np.exp(x - x.max(axis=2, keepdims=True))
            w /= w.sum(axis=2, keepdims=True)
            o = np.einsum("hgn,nhd->hgd", w, V)
            A = np.einsum("hgn,nhd->hgd", w, np.abs(V))
            e = (D * mass + 16 * (size + 1)) * 2.0 ** -24
            n = hi - lo
            lim = A * (2.0 ** -8 + 2 * e[..., None] + 2 * n * 2.0 ** -24) + 2.0 ** -8 * np.abs(o)
            out[t] = o.reshape(Hq, D)
            bound[t] = 1.1 * lim.reshape(Hq, D)
    return out, bound
