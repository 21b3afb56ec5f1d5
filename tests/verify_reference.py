"""The verification of drafted tokens by its definition in 64 bits (numpy),
one sequence and position after the other.  Shares no code with the library."""
import numpy as np


def probabilities(x, T):
    """Row of float64 logits -> its probabilities, or None where it has none."""
    if np.isnan(x).any() or (x == np.inf).any() or not np.isfinite(x).any() or not (T == 0 or 2.0 ** -20 <= T <= 2.0 ** 20):
        return None
    if T == 0:
        p = np.zeros_like(x)
        p[int(np.argmax(x))] = 1.0
        return p
    with np.errstate(over="ignore", under="ignore"):
        w = np.exp((x - x.max()) / T)
    return w / w.sum()


def verify(logits, sample_u, draft=None, accept_u=None, draft_probs=None, draft_len=None, temperature=None):
    """(tokens [B, L+1], accepted [B], probs [B, L+1], margin): margin is the
    least distance of a decision from its border: of the target from a step of the
    cumulative sum, in units of the probabilities' total, and of u q from p over
    the larger."""
    B = len(sample_u)
    L = 0 if draft is None else draft.shape[1]
    V = logits.shape[1]
    tokens, probs = np.full((B, L + 1), -1, np.int64), np.zeros((B, L + 1))
    accepted, margin = np.zeros(B, np.int64), np.inf
    for b in range(B):
        T = 1.0 if temperature is None else float(temperature[b])
        n = L if draft_len is None else min(max(int(draft_len[b]), 0), L)
        for j in range(n + 1):
            p = probabilities(logits[b * (L + 1) + j].astype(np.float64), T)
            accepted[b] = j
            if p is None:
                probs[b, j] = np.nan
                break
            w = p
            if j < n:
                t = int(draft[b, j])
                q = np.zeros(V)
                if draft_probs is not None:
                    q = draft_probs[b * L + j].astype(np.float64)
                elif 0 <= t < V:
                    q[t] = 1.0
                if 0 <= t < V:
                    lhs = float(accept_u[b, j]) * q[t]
                    if T > 0 and max(lhs, p[t]) > 0:
                        margin = min(margin, abs(lhs - p[t]) / max(lhs, p[t]))
                    if lhs < p[t]:
                        tokens[b, j], probs[b, j] = t, p[t]
                        continue
                w = np.maximum(p - q, 0.0)
                w = w if w.sum() > 0 else p
            cum = np.cumsum(w)
            target = float(sample_u[b]) * cum[-1]
            at = min(int(np.searchsorted(cum, target, side="right")), int(np.nonzero(w)[0][-1]))
            if T > 0:
                margin = min(margin, np.abs(cum - target).min())
            tokens[b, j], probs[b, j] = at, p[at]
            break
    return tokens, accepted, probs, margin
