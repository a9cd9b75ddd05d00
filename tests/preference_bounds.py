"""What float32 arithmetic leaves uncertain in a token's log probability and its
row of the gradient: bounds for each row by itself, from the entries that its
sum is made of.

u = 2^-24.  A row's sum of exp(x - max) has, relative to itself,
  2^-20           the exponentials: two approximate ones (2^-22 each) a term,
                  and the joins of threads and blocks,
  (chain + 64) u  additions: one thread's chain, and 64 to join the threads,
  3 u sum p |x - max|   the exponents' rounding, weighted as the terms are;
the logarithm and the subtractions add 4 u (lse - max) and 2 u |logp|.  The
size of the maximum itself is not in it: the log-sum-exp has two floats."""
import torch

U = 2.0 ** -24


def chain(vocab, dtype):
    """Terms in one thread: a warp takes rows of at most 16 KB, 256 threads
    longer ones."""
    return vocab / (32 if vocab * dtype.itemsize <= 16384 else 256)


def tokens(x, label):
    """(logps, their bounds, softmax, its bounds) of counted rows of logits."""
    kind = x.dtype
    x = x.double()
    top = x.amax(1, keepdim=True)
    near = torch.where(x > -torch.inf, x - top, 0.0)
    p = torch.softmax(x, 1)
    spread = torch.logsumexp(x - top, 1)
    at = torch.arange(x.shape[0], device=x.device)
    lp = (x[at, label] - top[:, 0]) - spread
    e = 2.0 ** -20 + (chain(x.shape[1], kind) + 64) * U + 3 * U * (p * near.abs()).sum(1) + 4 * U * spread
    # the gradient's exponents come from the log-sum-exp in one float, or where
    # that would be above 1024 from the row's maximum
    lse = top[:, 0] + spread
    e_soft = e + torch.where(lse.abs() < 1025, lse.abs(), spread) * U
    e_soft = p * (e_soft[:, None] + 2.0 ** -20 + 4 * U * (x - lse[:, None]).nan_to_num(0, 0, 0).abs().clamp_max(200))
    return lp, e + 2 * U * lp.abs(), p, e_soft
