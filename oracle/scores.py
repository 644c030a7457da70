"""Attention with score rules — dense float64, one request and one query head at a time.

Score of query head h at position p and key k: ``s = scale * q.k``, then
``softcap * tanh(s / softcap)``, then ``- slope_h * |p - k|``; key k is visible iff
``key_start <= k < min(L, max(p + 1, prefix_len))``; a query without visible keys gives zeros.
Keys and values come as each request's contiguous tensors, not through the page table."""
import math

import numpy as np


def paged_attention_scored(q, keys, values, query_start_loc, seq_lens, *, scale=None, softcap=0.0,
                           slopes=None, key_start=None, prefix_lens=None):
    """``q [N_pad, nh, hd]``, ``keys[i]``/``values[i] [L_i, nkv, hd]`` -> (out, weight) with
    ``weight = sum_k p_k |v_k|``, the scale of a rounding of every p_k."""
    q = np.asarray(q, np.float64)
    n_pad, nh, hd = q.shape
    scale = 1.0 / math.sqrt(hd) if scale is None else scale
    out = np.zeros((n_pad, nh, hd))
    weight = np.zeros((n_pad, nh, hd))
    for i, length in enumerate(int(x) for x in seq_lens):
        s0, s1 = int(query_start_loc[i]), int(query_start_loc[i + 1])
        if s1 == s0:
            continue
        pos = length - (s1 - s0) + np.arange(s1 - s0)
        key = np.arange(length)
        prefix = 0 if prefix_lens is None else int(prefix_lens[i])
        lo = np.zeros(s1 - s0, np.int64) if key_start is None else np.asarray(
            key_start[s0:s1], np.int64)
        hi = np.minimum(length, np.maximum(pos + 1, prefix))
        seen = (key[None, :] >= lo[:, None]) & (key[None, :] < hi[:, None])
        any_key = seen.any(axis=1)
        used = seen.any(axis=0)
        k64 = np.where(used[:, None, None], np.asarray(keys[i], np.float64), 0.0)
        v64 = np.where(used[:, None, None], np.asarray(values[i], np.float64), 0.0)
        nkv = k64.shape[1]
        for h in range(nh):
            kv = h // (nh // nkv)
            with np.errstate(invalid="ignore", over="ignore"):
                s = (q[s0:s1, h] @ k64[:, kv].T) * scale
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - float(slopes[h]) * np.abs(pos[:, None] - key[None, :])
            s = np.where(seen, s, -np.inf)
            m = np.where(any_key, s.max(axis=1, initial=-np.inf), 0.0)
            p = np.exp(s - m[:, None])
            z = p.sum(axis=1)
            p = p / np.where(any_key, z, 1.0)[:, None]
            # a key that a query does not see adds nothing, whatever its value holds
            v = v64[:, kv]
            if np.isfinite(v).all():
                out[s0:s1, h] = p @ v
                weight[s0:s1, h] = p @ np.abs(v)
            else:
                for j in range(s1 - s0):
                    out[s0 + j, h] = p[j, seen[j]] @ v[seen[j]]
                    weight[s0 + j, h] = p[j, seen[j]] @ np.abs(v[seen[j]])
    return out, weight
