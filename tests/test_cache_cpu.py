"""Refusals of the calls around the paged cache, on the host (fake, aligned device addresses; never dereferenced) and in
the Python wrappers (CPU tensors)."""
import ctypes

import numpy as np
import pytest
import torch

import kda_linear_attention_bounded_gb300 as kda
from kda_linear_attention_bounded_gb300 import build as kbuild

FAKE = 0x10000000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    from kda_linear_attention_bounded_gb300 import _binding
    return _binding.load()


def addresses(n, apart=0x1000000):
    """Places that are apart from each other."""
    return [FAKE + i * apart for i in range(n)]


def _rotary(lib, *, tokens=3, hq=4, hk=2, qs=512, ks=256, vs=256, os_=512, ps=3, num_axes=1, R=64, axes=None, mscale=1.0,
            kp=(2048, 256, 128), vp=(2048, 256, 128), pages=5, page=8, ws=None, ws_bytes=1024, **at):
    names = ("q", "k", "v", "positions", "slots", "freq", "k_pages", "v_pages", "out", "ws")
    a = dict(zip(names, addresses(len(names))))
    if ws is not None:
        a["ws"] = ws
    a.update(at)
    p = {n: P(v) for n, v in a.items()}
    return lib.kda_rotary_to_pages(p["q"], qs, p["k"], ks, p["v"], vs, tokens, hq, hk, p["positions"], ps, num_axes, p["slots"],
                                   p["freq"], R, None if axes is None else bytes(axes), 0, mscale, p["k_pages"], *kp, p["v_pages"],
                                   *vp, pages, page, p["out"], os_, p["ws"], ws_bytes, None)


def test_rotary_refusals(lib):
    for bad in (dict(tokens=-1), dict(hq=0), dict(hk=0), dict(hq=5000, qs=5000 * 128), dict(num_axes=0), dict(num_axes=5), dict(pages=-1),
                dict(page=0), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(positions=None), dict(slots=None),
                dict(freq=None), dict(q=FAKE + 2), dict(k=FAKE + 0x1000008), dict(positions=FAKE + 0x3000002),
                dict(slots=FAKE + 0x4000004), dict(freq=FAKE + 0x5000002), dict(qs=504), dict(qs=516), dict(ks=128), dict(vs=252),
                dict(os_=256), dict(num_axes=2, ps=2), dict(axes=[1] + [0] * 31), dict(num_axes=3, axes=[3] * 32),
                dict(kp=(2048, 256, 0)), dict(kp=(2048, 0, 128)), dict(kp=(64, 256, 128)), dict(vp=(2048, 256, 100)),
                dict(vp=(2048, 260, 128)), dict(k_pages=None), dict(v_pages=FAKE + 0x7000008)):
        assert _rotary(lib, **bad) == 1, bad
    for bad in (dict(R=0), dict(R=8), dict(R=72), dict(R=144), dict(mscale=float("nan")), dict(mscale=float("inf"))):
        assert _rotary(lib, **bad) == 2, bad
    for bad in (dict(ws=0), dict(ws=FAKE + 0x9000010), dict(ws_bytes=512)):
        assert _rotary(lib, **bad) == 3, bad
    assert _rotary(lib, tokens=0) == 0


def test_rotary_overlaps(lib):
    a = addresses(10)
    # out meets the keys, the values, the positions, the slots, the frequencies, or rows of q that are not its own
    for bad in (dict(out=a[1]), dict(out=a[2]), dict(out=a[3]), dict(out=a[4]), dict(out=a[5]), dict(out=a[0] + 512),
                dict(out=a[0], os_=520), dict(out=a[0], os_=1024)):
        assert _rotary(lib, **bad) == 1, bad
    # the pages meet an input or the output
    for bad in (dict(k_pages=a[0]), dict(v_pages=a[1]), dict(k_pages=a[8]), dict(v_pages=a[2] - 4096), dict(k_pages=a[3] - 16)):
        assert _rotary(lib, **bad) == 1, bad
    # q, k, v and out in one buffer of rows, out over the keys' columns
    one = dict(q=a[0], k=a[0] + 1024, v=a[0] + 1536, qs=1024, ks=1024, vs=1024, os_=1024)
    assert _rotary(lib, **one, out=a[0] + 1024 - 256) == 1
    assert _rotary(lib, **one, out=a[0] + 1024 + 256) == 1
    assert _rotary(lib, **one, out=a[0] - 256) == 1


def test_rotary_keys_on_values(lib):
    a = addresses(10)
    for off in (0, 16, 240, -16, -240):
        assert _rotary(lib, v_pages=a[6] + off) == 1, off
        assert _rotary(lib, v_pages=a[6] + off, pages=0, tokens=0) == 0


def _fork(lib, *, stride=8, width=8, B=4, forks=2, free=3, page=16, ws_bytes=1024, **at):
    names = ("table", "lens", "parents", "children", "free_pages", "src", "dst", "used", "ws")
    a = dict(zip(names, addresses(len(names))))
    a.update(at)
    p = {n: P(v) for n, v in a.items()}
    return lib.kda_fork_requests(p["table"], stride, width, p["lens"], B, p["parents"], p["children"], forks, p["free_pages"], free,
                                 page, p["src"], p["dst"], p["used"], p["ws"], ws_bytes, None)


def test_fork_refusals(lib):
    a = addresses(9)
    for bad in (dict(B=-1), dict(width=-1), dict(page=0), dict(stride=7), dict(forks=-1), dict(free=-1), dict(table=None), dict(lens=None),
                dict(parents=None), dict(children=None), dict(free_pages=None), dict(src=None), dict(dst=None), dict(used=None),
                dict(table=FAKE + 2), dict(lens=a[1] + 1), dict(parents=a[2] + 2), dict(used=a[7] + 1),
                # what is written meets an input, or each other
                dict(parents=a[0] + 8), dict(children=a[1]), dict(free_pages=a[5]), dict(src=a[6]), dict(used=a[1] + 4), dict(dst=a[0] + 16),
                dict(lens=a[0] + 3 * 32 + 28)):
        assert _fork(lib, **bad) == 1, bad
    for bad in (dict(ws=None), dict(ws=a[8] + 16), dict(ws_bytes=100)):
        assert _fork(lib, **bad) == 3, bad


def _release(lib, *, stride=8, width=8, B=4, rows=2, page=16, pages=9, ws_bytes=1024, **at):
    names = ("table", "lens", "rows", "free", "num", "ws")
    a = dict(zip(names, addresses(len(names))))
    a.update(at)
    p = {n: P(v) for n, v in a.items()}
    return lib.kda_release_requests(p["table"], stride, width, p["lens"], B, p["rows"], rows, page, p["free"], pages, p["num"], p["ws"],
                                    ws_bytes, None)


def test_release_refusals(lib):
    a = addresses(6)
    # (the parameter `rows` is the count, the pointer is named by its place)
    for bad in (dict(B=-1), dict(width=-1), dict(page=0), dict(stride=7), dict(pages=-1), dict(table=None), dict(lens=None),
                dict(free=None), dict(num=None), dict(table=FAKE + 2), dict(lens=a[1] + 1), dict(free=a[3] + 2), dict(num=a[4] + 2),
                dict(free=a[0]), dict(lens=a[2]), dict(num=a[3] + 32), dict(num=a[1]), dict(free=a[1] - 32)):
        assert _release(lib, **bad) == 1, bad
    for bad in (dict(ws=None), dict(ws=a[5] + 128), dict(ws_bytes=1023)):
        assert _release(lib, **bad) == 3, bad


def _compact(lib, *, stride=8, width=8, B=4, page=16, pages=9, new_stride=8, room=4, ws_bytes=1024, **at):
    names = ("table", "lens", "new", "src", "dst", "free", "num", "ws")
    a = dict(zip(names, addresses(len(names))))
    a.update(at)
    p = {n: P(v) for n, v in a.items()}
    return lib.kda_compact_pages(p["table"], stride, width, p["lens"], B, page, pages, p["new"], new_stride, p["src"], p["dst"], room,
                                 p["free"], p["num"], p["ws"], ws_bytes, None)


def test_compact_refusals(lib):
    a = addresses(8)
    for bad in (dict(B=-1), dict(width=-1), dict(page=0), dict(stride=7), dict(new_stride=5), dict(pages=-1), dict(room=3), dict(table=None),
                dict(lens=None), dict(new=None), dict(src=None), dict(dst=None), dict(free=None), dict(num=None), dict(new=a[2] + 2),
                dict(src=a[3] + 1), dict(dst=a[4] + 2), dict(free=a[5] + 3), dict(num=a[6] + 1),
                dict(new=a[0] + 4), dict(new=a[0], new_stride=9), dict(src=a[0] + 8), dict(dst=a[3]), dict(free=a[1]), dict(num=a[5]),
                dict(lens=a[2] + 32), dict(free=a[4] + 4)):
        assert _compact(lib, **bad) == 1, bad
    for bad in (dict(ws=None), dict(ws=a[7] + 1), dict(ws_bytes=0)):
        assert _compact(lib, **bad) == 3, bad


def _copy(lib, buffers=((0, 512, 512),), *, pages=6, count=2, ws_bytes=1024, **at):
    from kda_linear_attention_bounded_gb300._binding import PageBuffer
    a = dict(src=FAKE + 0x1000000, dst=FAKE + 0x2000000, ws=FAKE + 0x3000000)
    a.update(at)
    b = (PageBuffer * max(1, len(buffers)))(*(PageBuffer(None if x[0] is None else FAKE + x[0], *x[1:]) for x in buffers))
    return lib.kda_copy_pages(b, len(buffers), pages, P(a["src"]), P(a["dst"]), count, P(a["ws"]), ws_bytes, None)


def test_copy_refusals(lib):
    for bad in (dict(pages=-1), dict(count=-1), dict(src=None), dict(dst=None), dict(src=FAKE + 0x1000002), dict(dst=FAKE + 0x2000001),
                dict(buffers=[(None, 512, 512)]), dict(buffers=[(8, 512, 512)]), dict(buffers=[(0, 520, 512)]), dict(buffers=[(0, 512, 500)]),
                dict(buffers=[(0, 512, -16)]), dict(buffers=[(0, 256, 512)]), dict(buffers=[(0, 512, 512), (0, 512, 1 << 31)]),
                dict(src=FAKE + 512), dict(dst=FAKE + 5 * 512 + 508)):
        assert _copy(lib, **bad) == 1, bad
    for bad in (dict(ws=None), dict(ws=FAKE + 0x3000040), dict(ws_bytes=8)):
        assert _copy(lib, **bad) == 3, bad
    assert _copy(lib, count=0) == 0 and _copy(lib, pages=0) == 0 and _copy(lib, buffers=[]) == 0


def _prefix(lib, *, qs=512, kp=(2048, 256, 128), vp=(2048, 256, 128), pages=5, page=8, stride=8, width=8, B=4, T=2, groups=2, hq=4, hk=2,
            scale=0.1, os_=512, ws_bytes=None, **at):
    names = ("q", "k", "v", "table", "lens", "prefix", "starts", "out", "lse", "ws")
    a = dict(zip(names, addresses(len(names))))
    a.update(at)
    p = {n: P(v) for n, v in a.items()}
    if ws_bytes is None:
        ws_bytes = max(1024, lib.kda_shared_prefix_workspace_size(max(B, 0), max(T, 1), 4, 2, max(groups, 0)))
    return lib.kda_shared_prefix_attention(p["q"], qs, p["k"], *kp, p["v"], *vp, pages, page, p["table"], stride, width, p["lens"], B, T,
                                           p["prefix"], p["starts"], groups, hq, hk, scale, p["out"], os_, p["lse"], p["ws"], ws_bytes, None)


def test_shared_prefix_refusals(lib):
    a = addresses(10)
    for bad in (dict(B=-1), dict(T=0), dict(T=65), dict(hk=0), dict(hq=5), dict(hq=8192), dict(page=0), dict(pages=-1), dict(width=-1),
                dict(stride=7), dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(lens=None), dict(out=None),
                dict(q=FAKE + 8), dict(out=a[7] + 8), dict(lens=a[4] + 2), dict(lse=a[8] + 2), dict(qs=500), dict(os_=256),
                dict(kp=(2048, 256, 4)), dict(vp=(-8, 256, 128)), dict(groups=-1), dict(prefix=None), dict(starts=None),
                dict(prefix=a[5] + 2), dict(starts=a[6] + 1)):
        assert _prefix(lib, **bad) == 1, bad
    assert _prefix(lib, scale=float("nan")) == 2
    full = lib.kda_shared_prefix_workspace_size(4, 2, 4, 2, 2)
    for bad in (dict(ws=None), dict(ws=a[9] + 16), dict(ws_bytes=512), dict(ws_bytes=full - 1)):
        assert _prefix(lib, **bad) == 3, bad
    assert _prefix(lib, B=0) == 0


def test_shared_prefix_workspace(lib):
    size = lib.kda_shared_prefix_workspace_size
    assert size(-1, 1, 8, 2, 1) == 0 and size(4, 1, 8, 2, -1) == 0 and size(4, 0, 8, 2, 1) == 0 and size(4, 1, 8, 3, 1) == 0
    assert size(0, 1, 8, 2, 0) >= lib.kda_paged_workspace_size(8, 2, 1)
    for grown in ((8, 1, 8, 2, 1), (4, 2, 8, 2, 1), (4, 1, 16, 2, 1), (4, 1, 8, 2, 300)):
        assert size(*grown) > size(4, 1, 8, 2, 1), grown
    # rows of own tokens and of the pieces: each row of a group's key head twice at most, and 256 for each CTA
    rows = 192 * 32
    assert size(192, 1, 32, 4, 1) >= (rows * 528 + (rows + 152 * 256) * 544)


Z = torch.zeros(3, dtype=torch.int32)
WHOLE = {
    "page_size": [lambda n: kda.fork_requests(Z, Z, Z, Z, Z, n, copy_src=Z, copy_dst=Z, pages_used=Z, workspace=Z),
                  lambda n: kda.release_requests(Z, Z, Z, n, free_pages=Z, num_free=Z, workspace=Z),
                  lambda n: kda.compact_pages(Z, Z, n, new_table=Z, copy_src=Z, copy_dst=Z, free_pages=Z, num_free=Z, workspace=Z)],
    "T": [lambda n: kda.shared_prefix_attention(Z, Z, Z, Z, Z, Z, Z, n, out=Z, workspace=Z)],
}


@pytest.mark.parametrize("name", WHOLE)
def test_counts_are_whole_numbers(lib, name):
    for call in WHOLE[name]:
        for n in (2.9, 2.0, "16", None, np.float32(1), [1]):
            with pytest.raises(TypeError, match=f"{name}: expected a whole number"):
                call(n)
        for n in (2 ** 31, -2 ** 31 - 1, 2 ** 70):
            with pytest.raises(ValueError, match=f"{name}: out of range"):
                call(n)
        for n in (2, np.int64(2), True):
            with pytest.raises(ValueError, match="expected a CUDA tensor"):   # (the next check)
                call(n)


def test_axes_and_buffers_of_other_types(lib):
    with pytest.raises(TypeError):
        kda.rotary_to_pages(Z, Z, Z, Z, Z, Z, Z, Z, axes=[0.5], out=Z, workspace=Z)
    with pytest.raises(ValueError):
        kda.rotary_to_pages(Z, Z, Z, Z, Z, Z, Z, Z, axes=[300], out=Z, workspace=Z)
    with pytest.raises(TypeError, match="buffers: expected a list"):
        kda.copy_pages(Z, Z, Z, workspace=Z)
    with pytest.raises(ValueError, match="at least one"):
        kda.copy_pages([], Z, Z, workspace=Z)
    with pytest.raises(ValueError, match="buffers: expected a CUDA tensor"):
        kda.copy_pages([Z], Z, Z, workspace=Z)
    with pytest.raises(TypeError, match="buffers: expected a tensor"):
        kda.copy_pages([3], Z, Z, workspace=Z)
    with pytest.raises(TypeError):
        kda.shared_prefix_workspace_size(1, 1, 8, 2, 1.5)


def test_nothing_overlaps_in_shared_memory():
    """The hand-written map of the shared prefixes' kernel."""
    from test_shared_memory_cpu import constants
    known = constants("kda_prefix_attention.cu")
    value = lambda x: int(eval(str(x), {}, known))  # noqa: E731
    things = {"0": "kSlots * kTileBytes", "OFF_Q": "2 * kTileBytes", "OFF_MASK": "16 * kRing", "OFF_BAR": "8 * kBarriers",
              "OFF_ROWS": 2 * 128 * 4, "OFF_TMEM": 4, "OFF_ABORT": 4}
    spans = sorted((value(at), value(at) + value(size), at) for at, size in things.items())
    for (_, stop, a), (start, _, b) in zip(spans, spans[1:]):
        assert stop <= start, (a, b)
    assert spans[-1][1] + 1024 <= value("kSmemBytes") <= 227 * 1024   # (the map begins at a multiple of 1024)
    with open(f"{kbuild.CSRC}/kda_prefix_attention.cu") as f:
        text = f.read()
    # every barrier the kernel names lies among those counted
    assert "*turn = drained + 2;" in text and known["kBarriers"] == 2 * known["kSlots"] + 2 + 2 + 2 + 1 + 1 + 2 + 2
