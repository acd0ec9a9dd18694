"""flux_build_page_table against a host scheduler: block tables, slot map, positions."""
import numpy as np
import pytest
import torch

import q4_reference as ref
from sparse_attention_flux_b200.flux import (FLUX_ERR_DEVICE_CHECK, FLUX_ERR_INVALID_ARG,
                                             FLUX_ERR_SHAPE, FLUX_ERR_UNSUPPORTED, Context,
                                             FluxError)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    with Context(0, 16 << 20) as c:
        yield c


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Step:
    """One call's tensors: a table whose held pages came from the same free list."""

    def __init__(self, old, new, page, sink=0, window=0, spare=9, room=None, width=None, seed=0):
        g = np.random.default_rng(seed)
        cap = sink + window if window else 1 << 30
        need = sum(min(-(-n // page), cap) for n in new)
        self.free = g.permutation(need + spare)
        self.width = width or max(1, max(-(-n // page) for n in new)) + 2
        start = np.full((len(old), self.width), -7, np.int64)
        self.table, _, _, _, self.cursor = ref.page_table([0] * len(old), old, self.free, 0, start,
                                                          page, sink, window)
        total = sum(new) - sum(old)
        self.room = max(1, total if room is None else room)
        self.old, self.new, self.page, self.sink, self.window = old, new, page, sink, window
        self.t = dict(old=i32(old), new=i32(new), free=i32(self.free), cursor=i32([self.cursor]),
                      out=i32([-5]), table=i32(self.table),
                      slots=torch.full((self.room,), -9, dtype=torch.int64, device="cuda"),
                      pos=torch.full((self.room,), -9, dtype=torch.int32, device="cuda"),
                      cu=torch.full((len(old) + 1,), -9, dtype=torch.int32, device="cuda"))

    def run(self, ctx, **kw):
        t = self.t
        ctx.build_page_table(t["old"], t["new"], t["free"], t["cursor"], t["out"], t["table"],
                             t["slots"], t["pos"], self.page, self.sink, self.window,
                             cu_new=t["cu"], **kw)
        return self

    def want(self):
        return ref.page_table(self.old, self.new, self.free, self.cursor, self.table, self.page,
                              self.sink, self.window, self.room)

    def check(self):
        t = self.t
        for got, want, what in zip((t["table"], t["slots"], t["pos"], t["cu"], t["out"]),
                                   self.want(), ("table", "slots", "positions", "cu", "cursor")):
            assert np.array_equal(got.cpu().numpy().reshape(-1), np.asarray(want).reshape(-1)), what

    def check_refused(self):
        t = self.t
        assert np.array_equal(t["table"].cpu().numpy(), self.table)
        assert (t["slots"] == -1).all() and (t["pos"] == 0).all() and (t["cu"] == 0).all()
        assert t["out"].item() == self.cursor


@pytest.mark.parametrize("page", [16, 48, 64, 128])
@pytest.mark.parametrize("old,new", [
    ([0], [1]), ([0], [0]), ([5], [5]), ([63], [64]), ([64], [65]), ([15, 16, 17], [16, 17, 18]),
    ([0, 100, 0, 3], [1000, 100, 0, 777]), ([0] * 40, [1] * 40),
    (list(range(33)), [x * 3 for x in range(33)]),
])
@pytest.mark.parametrize("sink,window", [(0, 0), (1, 2), (0, 1), (2, 5)])
def test_small_steps(ctx, page, old, new, sink, window):
    Step(old, new, page, sink, window, room=sum(new) - sum(old) + 4).run(ctx).check()
    ctx.check()


@pytest.mark.parametrize("B", [1, 31, 32, 1023, 1025, 3000, 5200, 6120, 8192])
@pytest.mark.parametrize("window", [0, 3])
def test_many_requests(ctx, B, window):
    g = np.random.default_rng(B)
    old = g.integers(0, 90, B)
    new = old + g.integers(0, 50, B) * (g.random(B) < 0.7)
    Step(old.tolist(), new.tolist(), 16, 1 if window else 0, window, seed=B).run(ctx).check()
    ctx.check()


@pytest.mark.parametrize("window", [0, 17])
def test_long_prompts(ctx, window):
    Step([0, 131072, 70000, 0], [131072, 131073, 70000, 50001], 64, 2 if window else 0, window,
         room=190000).run(ctx).check()
    ctx.check()


def test_steps_in_a_row_in_place(ctx):
    """cursor_out is cursor: one buffer carries the free list through many steps."""
    g = np.random.default_rng(3)
    lens = np.array([0, 17, 200, 0, 64])
    s = Step(lens.tolist(), (lens + 600).tolist(), 32, spare=20)
    table, cursor, held = s.table, s.cursor, lens
    for step in range(12):
        new = held + g.integers(0, 50, 5)
        room = int((new - held).sum()) + 2
        slots = torch.empty(room, dtype=torch.int64, device="cuda")
        pos = torch.empty(room, dtype=torch.int32, device="cuda")
        ctx.build_page_table(i32(held), i32(new), s.t["free"], s.t["cursor"], s.t["cursor"],
                             s.t["table"], slots, pos, 32)
        table, want, wpos, _, cursor = ref.page_table(held, new, s.free, cursor, table, 32,
                                                      n_slots=room)
        assert np.array_equal(slots.cpu().numpy(), want) and np.array_equal(pos.cpu().numpy(), wpos)
        assert s.t["cursor"].item() == cursor
        held = new
    assert np.array_equal(s.t["table"].cpu().numpy(), table)
    ctx.check()


@pytest.mark.parametrize("case", ["shrinks", "negative", "too long", "slots", "pages", "cursor"])
def test_device_checks_hand_out_nothing(ctx, case):
    s = Step([10, 20, 0], [100, 90, 7], 16, spare=0,
             room=10 if case == "slots" else None, width=6 if case == "too long" else None) \
        if case != "too long" else Step([10, 20, 0], [96, 90, 7], 16, spare=0, width=6)
    if case == "shrinks":
        s.t["new"][1] = 19
    elif case == "negative":
        s.t["old"][2] = -1
    elif case == "too long":
        s.t["new"][0] = 97
    elif case == "pages":
        s.t["free"] = s.t["free"][:-1].contiguous()
    elif case == "cursor":
        s.cursor = len(s.free) + 1
        s.t["cursor"].fill_(s.cursor)
    s.run(ctx).check_refused()
    with pytest.raises(FluxError) as e:
        ctx.check()
    assert e.value.code == FLUX_ERR_DEVICE_CHECK
    ctx.check()


def test_sums_beyond_32_bits_are_refused(ctx):
    """Three requests of 2^30 tokens each: the sum of the new tokens wraps an int32."""
    s = Step([0, 0, 0], [5, 5, 5], 65536, width=20000)
    s.t["new"].fill_(1 << 30)
    s.run(ctx).check_refused()
    with pytest.raises(FluxError):
        ctx.check()


def test_negative_page_in_the_list(ctx):
    s = Step([0, 0], [40, 20], 16, spare=0)
    s.t["free"][1] = -3
    s.run(ctx)
    with pytest.raises(FluxError) as e:
        ctx.check()
    assert e.value.code == FLUX_ERR_DEVICE_CHECK
    _, slots, pos, _, _ = s.want()
    slots[16:32] = -1                       # the tokens of that page
    assert np.array_equal(s.t["slots"].cpu().numpy(), slots)
    assert np.array_equal(s.t["pos"].cpu().numpy(), pos)


def test_another_stream(ctx):
    st = torch.cuda.Stream()
    s = Step([0, 3], [300, 90], 16)
    st.wait_stream(torch.cuda.current_stream())
    s.run(ctx, stream=st)
    st.synchronize()
    s.check()


def test_binding_refuses_inconsistent_tensors(ctx):
    s = Step([0, 3], [300, 90], 16)
    good = dict(s.t)
    for key, bad, match in (("new", good["new"][:1], "inconsistent"),
                            ("pos", good["pos"][:-1], "inconsistent"),
                            ("slots", good["slots"].int(), "slots must be"),
                            ("cu", good["cu"][:2], "B \\+ 1"),
                            ("old", good["old"].cpu(), "CUDA"),
                            ("table", good["table"].t(), "contiguous")):
        s.t = dict(good, **{key: bad})
        with pytest.raises(ValueError, match=match):
            s.run(ctx)
    s.t = good
    for page, sink, window, code in ((24, 0, 0, FLUX_ERR_UNSUPPORTED), (16, 1, 0, FLUX_ERR_INVALID_ARG),
                                     (16, -1, 2, FLUX_ERR_INVALID_ARG)):
        s.page, s.sink, s.window = page, sink, window
        with pytest.raises(FluxError) as e:
            s.run(ctx)
        assert e.value.code == code
    assert FLUX_ERR_SHAPE == -2
