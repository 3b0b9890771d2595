"""Adjusted logits in float64: penalties for a row's history, biases, a mask.

y = x / r (x > 0) or x r where the token is in the history; y - (f c + p [c > 0]) with c its occurrences among
the made tokens (behind the prompt); y + the sum of its biases; -inf where the mask's bit is not set.
Ids outside [0, vocab) are not used.
"""

import numpy as np


def adjust_logits(x, history=None, history_len=None, prompt_len=None, repetition=None, frequency=None, presence=None,
                  bias_idx=None, bias=None, mask=None):
    x = np.array(x, np.float64)
    rows, vocab = x.shape
    for r in range(rows):
        if history is not None:
            n = history.shape[1] if history_len is None else min(max(int(history_len[r]), 0), history.shape[1])
            h = np.asarray(history[r][:n], np.int64)
            first = 0 if prompt_len is None else max(int(prompt_len[r]), 0)
            ok = (h >= 0) & (h < vocab)
            count = np.zeros(vocab)
            np.add.at(count, h[first:][ok[first:]], 1)
            with np.errstate(all="ignore"):
                if repetition is not None:
                    seen = np.unique(h[ok])
                    v, k = x[r, seen], float(repetition[r])
                    x[r, seen] = np.where(v > 0, v / k, v * k)
                f = 0.0 if frequency is None else float(frequency[r])
                p = 0.0 if presence is None else float(presence[r])
                x[r] = np.where(count > 0, x[r] - (f * count + p), x[r])
        if bias_idx is not None:
            ids = np.asarray(bias_idx[r], np.int64)
            ok = (ids >= 0) & (ids < vocab)
            add = np.zeros(vocab)
            np.add.at(add, ids[ok], np.asarray(bias[r], np.float64)[ok])
            x[r] += add
        if mask is not None:
            words = np.asarray(mask[r]).astype(np.int64) & 0xFFFFFFFF
            allowed = (words[np.arange(vocab) >> 5] >> (np.arange(vocab) & 31)) & 1
            x[r] = np.where(allowed == 1, x[r], -np.inf)
    return x
