"""The next step's page table built on a second stream while decode of the same ctx runs: the table
call's counter is its own, so both give what they give one after the other."""
import math

import pytest
import torch

from sparse_attention_flux_b200.flux import Context
from test_decode_q4 import Cache, normal
from test_page_table import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["4-bit", "bf16"])
def test_tables_and_decode_of_one_context(kv):
    with Context(0, 64 << 20) as ctx:
        # Row (0, 0), whose merge counts in the first word, is cut into many parts.
        lens = [30000, 64, 9000, 1]
        q = normal((4, 8, 128), 61)
        if kv == "4-bit":
            c = Cache(ctx, lens, 2, 128, 64, seed=60)
            decode = lambda st=None: c.decode(ctx, q, stream=st)  # noqa: E731
        else:
            k, v = normal((4, 30000, 2, 128), 62), normal((4, 30000, 2, 128), 63)
            sl = torch.tensor(lens, dtype=torch.int32, device="cuda")

            def decode(st=None):
                o, lse = torch.empty_like(q), torch.empty((4, 8), device="cuda")
                ctx.attn_decode(q, k, v, sl, o, 1 / math.sqrt(128), lse=lse, stream=st)
                return o, lse
        want = decode()
        steps = [Step([0, 131072, 70000, 0], [131072, 131073, 70000, 50001], 64, seed=i) for i in range(4)]
        for s in steps:
            s.run(ctx).check()
        torch.cuda.synchronize()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        for _ in range(5):
            got = []
            for s in steps:
                s.t["slots"].fill_(-9), s.t["out"].fill_(-5), s.t["table"].copy_(torch.as_tensor(s.table))
            torch.cuda.synchronize()
            for i in range(12):
                with torch.cuda.stream(a):
                    got.append(decode(a))
                if i % 3 == 0:
                    steps[i // 3].run(ctx, stream=b)
            torch.cuda.synchronize()
            for o, lse in got:
                assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
            for s in steps:
                s.check()
        ctx.check()
