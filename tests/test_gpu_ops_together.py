"""GPU: the rotary cache write, differential attention and compaction in one serving loop.

The native block manager drives prompts, decode steps, a fork with copy-on-write and an early end;
then the pool is compacted (K/V moved, the live block tables on the device renumbered) and decoding
goes on.  Every step's queries and new cache rows are checked against the float64 rotation, every
cached row of every live sequence against the row first written for it, bit for bit, and every
step's output against the float64 formula on those rows.
"""
import pytest
import torch

import paged_kv_cache_290_gb300 as pa
from paged_kv_cache_290_gb300 import binding as Bd
from paged_kv_cache_290_gb300.block_manager import BlockManager
from paged_kv_cache_290_gb300.workloads import PagedBatch, SeqSpec
from _diff_ref import diff_attention_ref
from test_gpu_rope import expect, rotated

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, NB, MB = 8, 4, 64, 16, 60, 12
AXES = pa.rope_axes([8, 12, 12])  # of 32 pairs: time, height, width


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_290_gb300 import build
    build.build()
    pa.load_library()
    assert torch.cuda.is_available()
    pa.get_device_error()


class Loop:
    def __init__(self, dtype, in_order):
        g = torch.Generator().manual_seed(7)
        self.dtype, self.in_order, self.g = dtype, in_order, g
        self.bm = BlockManager(NB, BS, prefix_caching=False)
        self.k = torch.full((NB, HKV, BS, D), float("nan"), dtype=dtype, device="cuda")
        self.v = self.k.clone()
        self.rows = {}  # sequence -> [(k, v)] of every token, as first written
        self.lam = 0.7 + 0.1 * torch.randn(HQ // 2, generator=g)
        self.weight = 1 + 0.1 * torch.randn(2 * D, generator=g)

    def step(self, new):
        """new: {sequence: tokens appended now}; the last step's tables if the manager kept them."""
        ids, lens = list(new), list(new.values())
        d = self.bm.descriptor(ids, lens, MB, device="cuda")
        t = sum(lens)
        qkv = torch.randn(t, (HQ + 2 * HKV) * D, generator=self.g).to(self.dtype).cuda()
        q, k, v = (x.view(t, -1, D) for x in qkv.split([HQ * D, HKV * D, HKV * D], 1))
        k0, v0, q0 = k.cpu(), v.cpu(), q.cpu()
        # a 4 x 6 image every 24 tokens: time, height and width positions
        at = torch.cat([torch.arange(len(self.rows.get(i, [])), len(self.rows.get(i, [])) + n)
                        for i, n in new.items()])
        pos = torch.stack((at // 24 + 1000, at // 6 % 4, at % 6))
        inv = pa.rope_inv_freq(D)
        pa.rope_and_cache(q, k, v, pos.cuda(), inv, self.k, self.v, d.slot_mapping, q_out=q, axes=AXES)
        yq, sq = rotated(q0, pos, inv, AXES, False, 1.0)
        expect(q.cpu(), yq, sq, self.dtype, 1.0)
        out = torch.full((t, HQ // 2, 2 * D), float("nan"), dtype=self.dtype, device="cuda")
        pa.diff_attention(q, self.k, self.v, d.block_tables, d.seq_lens, d.query_start_loc,
                          D ** -0.5, self.lam.cuda(), out, d.max_query_len, d.max_seq_len,
                          norm_weight=self.weight.cuda(), out_scale=0.4,
                          num_prefill_seqs=d.num_prefill_seqs)
        assert pa.get_device_error() == (0, 0)
        yk, sk = rotated(k0, pos, inv, AXES, False, 1.0)
        slots = d.slot_mapping.cpu()
        kc, vc = (c.cpu().transpose(1, 2).reshape(NB * BS, HKV, D) for c in (self.k, self.v))
        expect(kc[slots], yk, sk, self.dtype, 1.0)
        assert torch.equal(vc[slots], v0)
        row = 0
        for i, n in new.items():
            self.rows.setdefault(i, []).extend((kc[s], vc[s]) for s in slots[row:row + n])
            row += n
        self.check_cache(kc, vc)
        self.check_output(ids, lens, q.cpu(), out)
        return d

    def check_cache(self, kc, vc):
        for i, rows in self.rows.items():
            length, table = self.bm.sequence(i)
            assert length == len(rows)
            at = [table[p // BS] * BS + p % BS for p in range(length)]
            assert torch.equal(kc[at], torch.stack([k for k, _ in rows]))
            assert torch.equal(vc[at], torch.stack([v for _, v in rows]))

    def check_output(self, ids, lens, q, out):
        total = [len(self.rows[i]) for i in ids]
        b = PagedBatch(
            name="loop", num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, block_size=BS,
            scale=D ** -0.5, seqs=[SeqSpec(a, n) for a, n in zip(total, lens)],
            seq_lens=torch.tensor(total), query_start_loc=torch.tensor([0] + lens).cumsum(0),
            block_tables=None, q=q, k_new=None, v_new=None, slot_mapping=None, k_cache_pre=None,
            v_cache_pre=None, k_cache=self.k, v_cache=self.v, nan_block=-1, num_unique_blocks=0,
            k_contig=torch.cat([torch.stack([k for k, _ in self.rows[i]]) for i in ids]),
            v_contig=torch.cat([torch.stack([v for _, v in self.rows[i]]) for i in ids]),
            kv_start=torch.tensor([0] + total[:-1]).cumsum(0))
        ref, bound = diff_attention_ref(b, self.lam, self.weight, gain=0.4)
        assert torch.isfinite(out).all()
        assert ((out.cpu().double() - ref).abs() <= bound).all()

    def add(self, i, n):
        self.bm.add(i, list(range(n)))

    def append(self, i, n=1):
        pairs = self.bm.append(i, [5] * n)
        if pairs:
            Bd.copy_blocks(self.k, self.v, torch.tensor(pairs, dtype=torch.int32, device="cuda"))

    def compact(self, live):
        """Compacts; the live tables on the device are renumbered to what the manager then says."""
        old = torch.tensor([self.bm.sequence(i)[1] + [-1] * (MB - len(self.bm.sequence(i)[1]))
                            for i in live], dtype=torch.int32, device="cuda")
        moves = self.bm.compact(self.in_order)
        assert moves
        pa.move_blocks(self.k, self.v, moves, block_tables=old)
        assert pa.get_device_error() == (0, 0)
        for row, i in zip(old.tolist(), live):
            table = self.bm.sequence(i)[1]
            assert row == table + [-1] * (MB - len(table))


@pytest.mark.parametrize("in_order", [False, True], ids=["holes", "ordered"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_prompts_decoding_compaction_decoding(dtype, in_order):
    e = Loop(dtype, in_order)
    for i, n in ((1, 37), (2, 150), (3, 70), (4, 16)):
        e.add(i, n)
    e.step({1: 37, 2: 150, 3: 70, 4: 16})
    for i in (1, 2, 3, 4):
        e.append(i)
    e.step({1: 1, 2: 1, 3: 1, 4: 1})
    e.bm.fork(3, 5)  # shares every block; the next append copies the partial one
    e.rows[5] = list(e.rows[3])
    for i in (3, 5):
        e.append(i)
    e.step({3: 1, 5: 1})
    e.bm.free(2)
    del e.rows[2]
    e.compact([1, 3, 4, 5])
    e.add(6, 90)
    e.append(1, 3)
    e.append(5)
    e.step({5: 1, 6: 90, 1: 3})
    for i in (1, 3, 4, 5, 6):
        e.append(i)
    e.step({6: 1, 5: 1, 4: 1, 3: 1, 1: 1})
