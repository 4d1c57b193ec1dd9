"""Edges of the token-path calls that need no GPU to be seen."""
from __future__ import annotations

import os
import shutil
import subprocess
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import scan_stream_compaction_amd as ssc
from tests.sample_reference import sample_row
from tests.token_inputs import BLOCK_CASES, BLOCK_WIDTH, EQUAL_ROWS, block_case, group_sums

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "scan_stream_compaction_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")
def test_the_steps_over_the_most_assignments(tmp_path):
    """The row kernels take a token's `per` assignments in sets of 2, 4 or 8:
    the same steps on the host (tests/sets_walk.cpp), up to the largest `per`
    that the calls accept, under the sanitizer of signed overflow. An int that
    steps up by 8 passes its largest value from 2^31 - 7 assignments on."""
    exe = tmp_path / "sets_walk"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fsanitize=signed-integer-overflow",
                    "-fno-sanitize-recover=all", "-I", CSRC, os.path.join(HERE, "sets_walk.cpp"), "-o", str(exe)],
                   check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr


class _Device:
    """What torch.cuda.device does to the current device, without a GPU."""
    current = 0

    def __init__(self, device):
        self.device = device if isinstance(device, int) else device.index

    def __enter__(self):
        self.before, _Device.current = _Device.current, self.device

    def __exit__(self, *_):
        _Device.current = self.before


class _On:
    """A tensor's device, for a call that reads nothing else of it."""
    def __init__(self, index):
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.device.index


@pytest.mark.parametrize("at_record", [0, 1])
def test_a_prepared_row_call_runs_on_its_tensors_device(monkeypatch, at_record):
    """Called and repeated with the tensors' device current, whichever device
    is current at the time, and with the current one back afterwards."""
    ran = []

    class Lib:
        @staticmethod
        def ssc_dispatch_rows(*raw):
            ran.append((_Device.current, raw))
            return 0

    monkeypatch.setattr(_Device, "current", at_record)
    monkeypatch.setattr(ssc, "_lib", Lib)
    monkeypatch.setattr(ssc, "_current_device", lambda: _Device.current)
    monkeypatch.setattr(ssc, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(torch.cuda, "device", _Device)
    call = ssc.prepared(ssc._row_call, "ssc_dispatch_rows", _On(1), 5)
    for current in (0, 1, 2):
        _Device.current = current
        call()
        ssc._row_call("ssc_dispatch_rows", _On(1), 5)
        assert _Device.current == current
    assert ran == [(1, (5, 1001))] * 7


@pytest.mark.parametrize("n,vocab,hot", BLOCK_CASES)
def test_every_block_sum_shows(n, vocab, hot):
    """The inputs of the block sums' exact test: leaving out, doubling or
    exchanging any one block of 16, 256 or 4096 sorted positions of an id
    changes that id's sums, and no partial sum leaves fp32's whole numbers."""
    ids, rows = block_case(n, vocab, hot)
    assert 3 * n < 2 ** 24
    order = np.argsort(ids, kind="stable")
    key, rows = ids[order], rows[order]
    for size in (16, 256, 4096):
        m = n // size
        sums = rows[:m * size].reshape(m, size, BLOCK_WIDTH).sum(1, dtype=np.int64)
        whole = key[:m * size:size] == key[size - 1:m * size:size]
        assert bool((sums[whole] != 0).any(1).all())
        first = sums[whole]
        assert len(np.unique(first, axis=0)) == len(first)
    want = np.zeros((vocab, rows.shape[1]), np.int64)
    np.add.at(want, key, rows)
    assert np.array_equal(group_sums(key, rows, vocab), want)


@pytest.mark.parametrize("vocab,step,k,p,kept", [c for c in EQUAL_ROWS if c[0] <= 16_384])
def test_equal_weights_meet_the_border(vocab, step, k, p, kept):
    """The reference on equal logits: the count worked by hand, and one more
    where the comparison of the definition (less than) is taken as "or equal"."""
    x = np.where(np.arange(vocab) % step == 0, 0.5, -np.inf)
    for j in (0, 1, kept // 2, kept - 1):
        token, count, logprob = sample_row(x, j / kept, k=k, p=p)
        assert (token, count) == (j * step, kept) and abs(logprob + np.log(kept)) < 1e-12
    assert sample_row(x, 0.0, k=k, p=np.nextafter(p, 1))[1] == kept + 1


def test_the_series_of_the_weights():
    """2^r on [-1/2, 1/2] by the eleven terms that the sampling kernel takes:
    within 8.7e-15 of itself, and with some 2^-53 of the argument and the steps
    under the 2^-46 of the largest weight that include/ssc.h states."""
    with localcontext() as ctx:
        ctx.prec = 40
        ln2 = Decimal(2).ln()

        def off(r):
            term = total = Decimal(1)
            for k in range(1, 12):
                term = term * ln2 * r / k
                total += term
            return abs(total / (ln2 * r).exp() - 1)
        worst = max(off(Decimal(i) / 1000) for i in range(-500, 501))
        assert Decimal("8.6e-15") < worst < Decimal("8.7e-15")
        # weight 2^y: rate, product and Horner's steps off by up to 4 and 3 of 2^-53
        total = max(Decimal(2) ** y * (worst + (4 * -y * ln2 + 3) * Decimal(2) ** -53)
                    for y in (Decimal(i) / 100 for i in range(-5000, 1)))
        assert total < Decimal(2) ** -46
