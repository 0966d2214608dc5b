"""Every tile that the grouped products choose, with plans whose tiles are whole and split, on an MI355X, against 64-bit values."""
import functools
import os
import re

import numpy as np
import pytest

import workloads as wl
from tests import operator_values as ov
from tests.test_gpu_grouped import assert_close, env, expect, experts  # noqa: F401

FORMATS = ["q8_0", "q4_0", "q4_1", "q4_k", "q6_k"]
CUS = 256


def up(a, b):
    return -(-a // b)


def tile_of(wide_x, fmt, items, E, matrix_rows):
    """(tokens of a tile, waves that share rows, parts of a plan's tile, whether its row tiles take more than one unit)."""
    tile = 128 if items >= 48 * E else 32
    groups, wide = min(E, items), 64 if wide_x else 128
    each = items // groups
    if tile == 128 and groups * up(each, wide) * up(matrix_rows, 128) >= CUS:
        return wide, 1, tile // wide, up(matrix_rows, 128) > 32
    waves = groups * up(each, 32) * up(matrix_rows, 32)
    # workgroups of two waves to a row that a compute unit holds
    two = (1 if fmt in ("q8_0", "q6_k") else 2) if wide_x else 2 if fmt == "q8_0" else 3
    if wide_x:
        kg = 4 if waves <= CUS else 2 if (waves < 8 * CUS if two > 1 else waves <= 2 * CUS) else 1
    else:
        kg = 8 if waves <= CUS else 4 if waves <= 2 * CUS else 2 if waves <= 2 * two * CUS else 1
    return 32, kg, tile // 32, up(matrix_rows, 128 // min(kg, 4)) > 32


# items, experts, matrix rows
CASES = [(120, 2, 1100), (180, 3, 2100), (128, 2, 4200), (600, 6, 4200), (520, 4, 8300), (30, 1, 1100), (90, 4, 2700), (90, 4, 6300),
         (200, 8, 8300), (300, 1, 33100)]
SHAPES = {False: {(128, 1, 1), (32, 1, 1), (32, 2, 1), (32, 4, 1), (32, 8, 1), (32, 1, 4), (32, 2, 4), (32, 4, 4), (32, 8, 4)},
          # one wave to 32 rows takes 2048 waves where a compute unit holds two workgroups of two waves to a row: split tiles
          # have as many workgroups of 64 tokens then
          True: {(64, 1, 2), (32, 1, 1), (32, 2, 1), (32, 4, 1), (32, 2, 4), (32, 4, 4)}}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("wide_x", [False, True])
def test_the_cases_take_every_tile(wide_x, fmt):
    got = {tile_of(wide_x, fmt, *c) for c in CASES}
    want = SHAPES[wide_x]
    if wide_x and fmt in ("q8_0", "q6_k"):
        want = want | {(32, 1, 4)}
    assert {g[:3] for g in got} == want
    assert {g[1] for g in got if g[2] > 1 and g[3]} == {k for _, k, split in want if split > 1}


def test_the_rule_is_the_sources():
    """tile_of() follows launch_tile_n and plan_tile: where these change, so has it, and the cases with it."""
    root = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bandwidth_bound_block_amd", "csrc")
    src = open(os.path.join(root, "qmv_tile.h")).read()
    body = re.sub(r"//[^\n]*", "", src[src.index("int32_t launch_tile_n("):src.index("int32_t launch_tile_x(")])
    said = [" ".join(m.split()) for m in re.findall(r"if \(((?:[^()]|\([^()]*\))*)\)\s*return launch_tile_s<F, XT, (?:\w+, \d+)>", body)]
    assert said == ["tile == 128 && wide >= cus", "waves <= cus && near", "kTwo > 1 ? waves < 8 * cus : waves <= 2 * cus",
                    "waves <= cus && near", "waves <= 2 * cus && near", "waves <= 2 * kTwo * cus"], said
    assert re.findall(r"return launch_tile_s<F, XT, (\w+, \d+)>", body) == ["kWide, 1", "32, 4", "32, 2", "32, 8", "32, 4", "32, 2", "32, 1"]
    assert "kTwo = TileShape<F, XT, 32, 2>::kWgs;" in body
    assert "kWgs = std::min(4 * kOcc / kWaves, kLdsMax / (kLds + 1024));" in src
    assert "kWideX ? 64 : 128" in body
    assert "constexpr int kRowGroup = 32;" in src
    group = open(os.path.join(root, "qmv_group.hip")).read()
    assert "return n_items >= 48 * (int64_t)n_groups ? 128 : 32;" in group


def routing(items, E):
    """Uneven: the first group over a tile of 128 where there are so many, some with few items or (of more than two) none."""
    g = np.random.default_rng(items + E)
    p = np.arange(E, 0, -1.0)
    if E > 2:
        p[1] = 0.0
        p[2] = 0.05
    return g.choice(E, size=(items, 1), p=p / p.sum())


@functools.lru_cache(maxsize=1)
def values(fmt, items, E, rows):
    K = 512 if fmt in ("q4_k", "q6_k") else 288
    W = experts(fmt, f"t/shapes/{fmt}/{rows}", E, rows, K)
    ids = routing(items, E)
    x = np.random.default_rng(rows).standard_normal((items, K))
    import torch
    xt, x = ov.as_type(torch, x, "bf16")            # values of fp32 as they are
    return W, ids, xt, expect(fmt, W[2], rows, K, ids, x)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("items,E,rows", CASES)
@pytest.mark.parametrize("x_name", ["bf16", "f32"])
def test_tiles(env, fmt, items, E, rows, x_name):  # noqa: F811
    torch, qmv = env
    print("tiles", fmt, x_name, items, E, rows, tile_of(x_name == "f32", fmt, items, E, rows), flush=True)
    (buf, stride, W), ids, xt, (y, e) = values(fmt, items, E, rows)
    K = xt.shape[1]
    x = (xt.float() if x_name == "f32" else xt).cuda()
    plan = qmv.qmv_group_plan(torch.from_numpy(ids.astype(np.int32)).cuda(), E)
    got = qmv.qmv_moe_grouped(fmt, torch.from_numpy(buf).cuda(), stride, E, rows, K, plan, 1, x)
    assert_close(got, y, e, fmt)
    # the same rows as gate and up
    if rows % 2 == 0:
        F = rows // 2
        h, eh = ov.swiglu(y[..., :F], e[..., :F], y[..., F:], e[..., F:])
        got = qmv.qmv_moe_grouped_swiglu(fmt, torch.from_numpy(buf).cuda(), stride, E, F, K, plan, 1, x)
        assert_close(got, h, eh, fmt)
