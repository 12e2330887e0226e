"""Penalties, biases and an allowed-token mask on logits, restated on the CPU in
float64, entry by entry.

Test infrastructure only (see the package docstring).
"""
from __future__ import annotations

import math

import numpy as np


def _row(x, tokens, n_prompt, rep, pres, freq, biases, allowed):
    """One row; `biases` a list of (token, value), `allowed` a list of bools."""
    x = [float(v) for v in x]
    vocab = len(x)
    spread = [abs(v) for v in x]                # magnitudes added up, for error bounds
    for i in range(vocab):
        seen = any(t == i for t in tokens)
        count = sum(1 for t in tokens[n_prompt:] if t == i)
        if seen:
            x[i] = x[i] / rep if x[i] > 0 else x[i] * rep
            spread[i] = abs(x[i])
        if count:
            x[i] -= freq * count
            x[i] -= pres
            spread[i] += abs(freq) * count + abs(pres)
        mine = [w for t, w in biases if t == i]
        if mine:
            x[i] += mine[-1]
            spread[i] += abs(mine[-1])
        if not allowed[i]:
            x[i] = -math.inf
    return x, spread


def apply(logits, token_ids=None, prompt_lens=None, token_lens=None, repetition=None,
          presence=None, frequency=None, bias_offsets=None, bias_ids=None, bias_values=None,
          allowed_mask=None):
    """(B, V) float64 results and the (B, V) sums of the magnitudes that went into
    each.  Lists a row may not use (ids outside the vocabulary) are dropped."""
    logits = np.asarray(logits, np.float64)
    B, V = logits.shape
    out, spread = np.empty((B, V)), np.empty((B, V))
    for b in range(B):
        tokens, n_prompt = [], 0
        if token_ids is not None:
            n = int(token_lens[b]) if token_lens is not None else token_ids.shape[1]
            p = int(prompt_lens[b]) if prompt_lens is not None else 0
            if 0 <= p <= n <= token_ids.shape[1]:
                tokens, n_prompt = [int(t) for t in token_ids[b, :n]], p
        rep = float(repetition[b]) if repetition is not None else 1.0
        pres = float(presence[b]) if presence is not None else 0.0
        freq = float(frequency[b]) if frequency is not None else 0.0
        rep = rep if math.isfinite(rep) and rep > 0 else 1.0
        pres = pres if math.isfinite(pres) else 0.0
        freq = freq if math.isfinite(freq) else 0.0
        biases = []
        if bias_offsets is not None:
            a, e = int(bias_offsets[b]), int(bias_offsets[b + 1])
            if 0 <= a <= e <= len(bias_ids):
                biases = list(zip(bias_ids[a:e].tolist(), bias_values[a:e].tolist()))
        allowed = [True] * V
        if allowed_mask is not None:
            allowed = [bool(int(allowed_mask[b, i // 32]) >> (i % 32) & 1) for i in range(V)]
        out[b], spread[b] = _row(logits[b], tokens, n_prompt, rep, pres, freq, biases, allowed)
    return out, spread
