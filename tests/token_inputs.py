"""Inputs whose results are exact, so that a call's are compared for equality:
small whole numbers as rows, and equal logits as weights."""
from __future__ import annotations

import numpy as np

# tokens, vocabulary, share of the tokens that have id 0: with one, two or
# three levels of block sums and several blocks of the largest
BLOCK_CASES = [(255, 1, 0.0), (4111, 2, 0.5), (70_001, 1, 0.0), (70_001, 3, 0.9), (262_143, 1, 0.0), (300_007, 1, 0.0),
               (300_007, 3, 0.9), (300_007, 5, 0.0), (2_500_009, 2, 0.8)]
BLOCK_WIDTH = 24


def block_case(n, vocab, hot):
    """(ids, rows): rows of whole numbers of [-3, 3]: sums of up to 5,592,405
    of them stay below 2^24, so that fp32 holds every partial sum."""
    r = np.random.RandomState(n + vocab)
    ids = np.where(r.rand(n) < hot, 0, r.randint(0, vocab, n))
    return ids, r.randint(-3, 4, (n, BLOCK_WIDTH)).astype(np.int8)


def group_sums(ids, rows, vocab):
    """Sums of rows by id, as int64."""
    order = np.argsort(ids, kind="stable")
    ends = np.cumsum(np.bincount(ids, minlength=vocab))
    run = np.concatenate([np.zeros((1, rows.shape[1]), np.int64), np.cumsum(rows[order], axis=0, dtype=np.int64)])
    return run[ends] - run[np.concatenate([[0], ends[:-1]])]


# Equal logits all weigh 1, so that with a share of 1/4, 1/2 or 3/4 the running
# weight meets top_p times the sum exactly: the tokens before the border are
# kept, the one at it is not. Rows of: vocabulary, every step-th logit a token
# (the others masked), top_k, top_p, kept.
EQUAL_ROWS = [(vocab, step, k, p, int((min(k, vocab // step) if k else vocab // step) * p))
              for vocab in (64, 4096, 16_384, 131_072)
              for step in (1, 2)
              for k in (0, 32, 2048, 4096, 65_536)
              for p in (0.25, 0.5, 0.75)]
