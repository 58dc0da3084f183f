"""The ring of tiles that the norm's checkpoint kernels read through, when a wait for a copy gives
up: no copy may still be in flight when the CTA leaves, and no time is spent on barriers that
nothing will complete. On simulated barriers here, and on the GPU with a copy left out."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "nvfp4_block_scaled_quantize_gb300", "csrc")
OUT = os.path.join(HERE, "probes", "_build")
LIMIT = 100  # of a simulated wait


def _compile(source, command):
    os.makedirs(OUT, exist_ok=True)
    lib = os.path.join(OUT, "lib%s.so" % os.path.splitext(source)[0])
    tmp = "%s.%d" % (lib, os.getpid())
    r = subprocess.run([*command, "-std=c++17", "-shared", "-I", CSRC,
                        os.path.join(HERE, "probes", source), "-o", tmp],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    os.replace(tmp, lib)
    return ctypes.CDLL(lib)


@pytest.fixture(scope="module")
def sim():
    L = _compile("tile_ring_sim.cpp", ["g++", "-O2", "-Wall", "-Werror", "-fPIC"])

    def run(stages, delay):
        d = np.asarray(delay, np.int64)
        out = np.zeros(5, np.int64)
        assert L.tile_ring_sim(stages, len(d), ctypes.c_void_p(d.ctypes.data),
                               ctypes.c_void_p(out.ctypes.data)) == 0
        return dict(zip(("gave_up", "in_flight", "timeouts", "idle", "wrong"), out.tolist()))
    return run


@pytest.mark.parametrize("stages", [1, 2, 3, 4])
def test_every_tile_is_read_in_its_turn(sim, stages):
    rng = np.random.default_rng(stages)
    for tiles in (1, 2, 3, 4, 5, 17, 64):
        r = sim(stages, rng.integers(0, LIMIT, tiles))
        assert r == dict(gave_up=-1, in_flight=0, timeouts=0, idle=0, wrong=0), (tiles, r)


@pytest.mark.parametrize("stages", [1, 2, 3, 4])
def test_nothing_is_in_flight_after_a_wait_that_gave_up(sim, stages):
    """One late tile, which lands after the wait for it has given up and before a second limit,
    with any number of tiles after it: whole and half turns of the ring."""
    for tiles in range(1, 20):
        for late in range(tiles):
            for after in (0, LIMIT // 2):
                delay = np.zeros(tiles, np.int64)
                # fetched at the same time as it or later, and landing after it
                delay[late + 1:] = after
                delay[late] = LIMIT + LIMIT // 2
                r = sim(stages, delay)
                assert r == dict(gave_up=late, in_flight=0, timeouts=1, idle=0,
                                 wrong=0), (tiles, late, r)


@pytest.mark.parametrize("stages", [1, 2, 3, 4])
def test_later_copies_that_outlast_the_lost_one_are_waited_for(sim, stages):
    """A tile that never lands, and the tiles fetched with it landing only during the drain: the
    lost copy alone is left, and only its own two waits run out."""
    for tiles in range(1, 20):
        for lost in range(tiles):
            delay = np.zeros(tiles, np.int64)
            delay[lost + 1:] = 2 * LIMIT + LIMIT // 2
            delay[lost] = -1
            r = sim(stages, delay)
            assert r == dict(gave_up=lost, in_flight=1, timeouts=2, idle=0,
                             wrong=0), (tiles, lost, r)


@pytest.mark.gpu
@pytest.mark.parametrize("stages", [1, 2, 3, 4])
def test_a_copy_that_never_comes(stages):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.init()
    L = _compile("tile_ring_probe.cu", ["nvcc", "-gencode", "arch=compute_103a,code=sm_103a", "-O3",
                                        "-Xcompiler", "-fPIC"])
    vp = ctypes.c_void_p
    L.probe_tile_ring.argtypes = [ctypes.c_int] * 3 + [vp] * 4
    dev = torch.device("cuda")
    for tiles in (1, 3, 9, 14):
        src = torch.arange(tiles * 64, dtype=torch.int32, device=dev)
        for dropped in sorted({-1, 0, tiles // 2, tiles - 1}):
            seen = torch.zeros(tiles, 64, dtype=torch.int32, device=dev)
            info = torch.zeros(4, dtype=torch.int32, device=dev)
            assert L.probe_tile_ring(stages, tiles, dropped, src.data_ptr(), seen.data_ptr(),
                                     info.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
            gave_up, issued, landed, threads = info.tolist()
            read = tiles if dropped < 0 else dropped
            assert torch.equal(seen[:read], src.view(tiles, 64)[:read])
            assert bool((seen[read:] == -1).all())
            assert gave_up == dropped and threads == (0 if dropped < 0 else 64)
            # the owner stops fetching where it gives up
            ahead = max(stages - 1, 1)
            assert issued == (tiles if dropped < 0 else min(tiles, dropped + ahead) - 1)
            assert landed == issued
