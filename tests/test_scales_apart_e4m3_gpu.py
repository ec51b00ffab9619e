"""The attention step over a cache in 8 bits where keys of the largest scores have values whose scale lies far below
the others' (blocks of zeros have 2^-126): sums of weights in units of a scale stay in range.  Tolerances of
tests/test_decode_e4m3_gpu.py, and 2^-126 for what is too small for an output."""
import math

import pytest
import torch

import test_decode_e4m3_gpu as base
from oracle import rollout_oracle as ro
from shared_prefix_grouped_gb300 import api
from test_decode_e4m3_gpu import built  # noqa: F401  (the build, before anything here)

pytestmark = pytest.mark.gpu
E = base.E


def steep(plens, olens, zeros, gap, again=None, d=128, hq=8, hk=2, scale=2.0 ** -126):
    """Scores of gap ln 2 where the values are zeros (key ranges of the prefix and of the own keys), 0 elsewhere;
    a quarter more in the range `again`, of ordinary values."""
    p = base.problem(plens, [len(olens)], olens, hq, hk, d, 16, torch.bfloat16, seed=gap)
    p["q"][:] = 0
    p["q"][:, :, 0] = gap * math.log(2)
    p["q"][:, 1::2, 0] *= 0.97                # (heads of other maxima)
    k, v = p["codes"]
    ks, vs = p["scales"]
    live = ~k.isnan()
    k[..., 0] = torch.where(live[..., 0], torch.zeros_like(k[..., 0]), k[..., 0])

    def blocks(where, keys):
        rows = [p["pp"][0]] if where == "prefix" else list(p["op"])
        n = [plens[0]] if where == "prefix" else olens
        return [int(row[i // 16]) for row, m in zip(rows, n) for i in range(*keys, 16) if i < m]

    for where, keys, level in [(*z, 256.0) for z in zeros] + ([(*again, 320.0)] if again else []):
        for page in blocks(where, keys):
            ks[page] = 2.0 ** -8
            k[page, :, :, 0] = torch.where(live[page, :, :, 0], torch.full_like(k[page, :, :, 0], level),
                                           k[page, :, :, 0])
            if level == 256.0:
                v[page] = torch.where(live[page], torch.zeros_like(v[page]) if scale == 2.0 ** -126 else v[page], v[page])
                vs[page] = scale
    return p


def check(p, o, lse, tensor_cores=True):
    ref, rl, mass, least, A, W = ro.decode_e4m3(p["q"], p["codes"], p["scales"], p["plens"], p["gsizes"], p["pp"],
                                                p["op"], p["olens"] if p["wo"] else None, 1.0)
    K = max(p["plens"]) + int(p["olens"].max()) + 1
    sums = (K / 8 + 64) * E
    score = (p["q"].shape[2] + 4) * E * A + (2.0 ** -17 * W if tensor_cores else 0)
    tol = (2 * score + sums + (2.0 ** -7 if tensor_cores else 0)) * mass + least + 2.0 ** -8 * ref.abs() + 2.0 ** -126
    o, lse = o.cpu().double(), lse.cpu().double()
    assert bool(((lse - rl).abs() <= score + sums + 4 * E * rl.abs()).all()), float((lse - rl).abs().max())
    assert bool(((o - ref).abs() <= tol).all()), float(((o - ref).abs() - tol).max())
    assert api.device_status() == 0


RANGES = [("prefix", (0, 128)), ("prefix", (0, 64)), ("prefix", (64, 128)), ("prefix", (0, 16)), ("prefix", (128, 256)),
          ("prefix", (0, 512)), ("prefix", (0, 992)), ("own", (0, 32)), ("own", (0, 16)), ("own", (0, 64)),
          ("own", (32, 64)), ("own", (0, 288))]


@pytest.mark.parametrize("gap", [100, 119, 150, 200])
@pytest.mark.parametrize("zeros", RANGES, ids=lambda z: f"{z[0]}{z[1][0]}-{z[1][1]}")
def test_zeros_outweigh_what_follows(zeros, gap):
    for plens, olens in (([1000], [300, 5]), ([1000], [0, 0]), ([0], [300, 7])):
        if (zeros[0] == "prefix") == (plens[0] == 0) or (zeros[0] == "own") == (olens[0] == 0):
            continue
        p = steep(plens, olens, [zeros], gap, d=64 if gap == 119 else 128)
        check(p, *base.run(p, scale=1.0))
        check(p, *base.run(p, flags=base.SIMT, scale=1.0), tensor_cores=False)


@pytest.mark.parametrize("gap", [100, 120, 160])
@pytest.mark.parametrize("place", ["prefix", "own"])
def test_and_are_outweighed_in_turn(place, gap):
    # the sum's unit, held back by the zeros, catches up when a larger score has made them negligible
    n = 992 if place == "prefix" else 512
    for again in ((n - 16, n), (256, 272), (320, 336)):
        p = steep([1000] if place == "prefix" else [0], [300, 5] if place == "prefix" else [512, 40], [(place, (0, 128))],
                  gap, again=(place, again))
        check(p, *base.run(p, scale=1.0))


@pytest.mark.parametrize("place", ["prefix", "own"])
def test_many_query_heads(place):
    # two groups of eight rows in the own-key kernel
    p = steep([1000], [300, 65], [(place, (0, 64))], 130, hq=16, hk=1)
    check(p, *base.run(p, scale=1.0))


@pytest.mark.parametrize("place", ["prefix", "own"])
def test_small_values_that_outweigh(place):
    # within 2^-118 of the others' scale values count as they are, though their weight is 2^110 of the others'
    for scale in (2.0 ** -60, 2.0 ** -100):
        p = steep([1000], [300, 65], [(place, (0, 128))], 110, scale=scale)
        check(p, *base.run(p, scale=1.0))
