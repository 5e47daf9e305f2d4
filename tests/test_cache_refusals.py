"""What the calls on the paged cache refuse on the host (no GPU: the checks touch
no device state), and how attention's work is split."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40  # an address that is never dereferenced


@pytest.fixture(scope="module")
def B():
    from draft_verification_amd import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding


@pytest.fixture(scope="module")
def cfg(B):
    return B.Config(8, 8, 1000, B.SV_BF16, 0)


def cache(B, **more):
    d = dict(n_slots=8, n_pages=100, page_size=16, max_pages=10, page_table=FAKE, lengths=FAKE, page_counts=FAKE,
             page_refs=FAKE, free_pages=FAKE)
    d.update(more)
    return B.make_cache(**d)


def kv(B, **more):
    d = dict(kv_heads=2, head_dim=64, type=B.SV_KV_BF16, keys=FAKE, values=FAKE, strides=(2048, 1024, 64))
    d.update(more)
    return B.make_kv(**d)


BAD_CACHES = [dict(n_slots=0), dict(n_pages=0), dict(page_size=0), dict(page_size=24), dict(page_size=2048),
              dict(max_pages=0), dict(max_pages=1 << 27), dict(n_pages=(1 << 24) + 1), dict(page_table=None),
              dict(lengths=None), dict(n_slots=1 << 20)]
BAD_KVS = [dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=0), dict(head_dim=72), dict(head_dim=272), dict(type=2),
           dict(keys=None), dict(values=None), dict(keys=FAKE + 8), dict(values=FAKE + 2), dict(strides=(32, 1024, 64)),
           dict(strides=(2048, 1028, 64)), dict(strides=(2048, 1024, 56)), dict(strides=(2048, 1024, 68)),
           dict(type=1, strides=(2048, 1024, 72))]


def refused(status, B):
    return status in (B.SV_EINVAL, B.SV_EUNSUPPORTED)


@pytest.mark.parametrize("kind", range(6))
def test_pages_accepts(B, cfg, kind):
    a = B.make_pages_args(4, kind=kind, cache=cache(B), slots=FAKE, from_slots=FAKE, rows=5, granted=FAKE, copies=FAKE,
                          max_copies=4)
    assert B.pages_check(cfg, a) == B.SV_OK
    a.B = 0
    assert B.pages_check(cfg, a) == B.SV_OK


@pytest.mark.parametrize("kind", range(6))
@pytest.mark.parametrize("more", BAD_CACHES + [dict(page_counts=None), dict(page_refs=None), dict(free_pages=None)])
def test_pages_refuses_caches(B, cfg, kind, more):
    a = B.make_pages_args(4, kind=kind, cache=cache(B, **more), slots=FAKE, from_slots=FAKE, rows=5, granted=FAKE,
                          copies=FAKE, max_copies=4)
    assert refused(B.pages_check(cfg, a), B)


@pytest.mark.parametrize("kind,field,value", [
    (1, "B", -1), (1, "B", 9), (1, "rows", -1), (1, "rows", (1 << 30) + 1), (2, "rows", -1), (3, "B", 9),
    (4, "granted", None), (4, "from_slots", None), (4, "copies", None), (4, "max_copies", 3), (5, "copies", None),
    (4, "copies", FAKE + 4), (5, "copies", FAKE + 4),
    (5, "max_copies", -1), (5, "max_copies", (1 << 24) + 1), (1, "kind", 6), (1, "kind", -1),
])
def test_pages_refuses(B, cfg, kind, field, value):
    a = B.make_pages_args(4, kind=kind, cache=cache(B), slots=FAKE, from_slots=FAKE, rows=5, granted=FAKE, copies=FAKE,
                          max_copies=4)
    setattr(a, field, value)
    assert refused(B.pages_check(cfg, a), B)


def test_pages_without_slots_needs_one_for_each_sequence(B, cfg):
    a = B.make_pages_args(4, kind=B.SV_PAGES_RELEASE, cache=cache(B, n_slots=3))
    assert B.pages_check(cfg, a) == B.SV_EINVAL
    big = B.Config(5000, 8, 1000, B.SV_BF16, 0)
    a = B.make_pages_args(4097, kind=B.SV_PAGES_RELEASE, cache=cache(B, n_slots=5000))
    assert B.pages_check(big, a) == B.SV_EUNSUPPORTED


@pytest.mark.parametrize("field,value,fine", [
    ("n_copies", 0, True), ("n_copies", -1, False), ("copies", None, False), ("pools", None, False), ("pools", FAKE + 8, False),
    ("copies", FAKE + 4, False), ("n_pools", 0, False), ("n_pools", 65536, False), ("n_pools", 1, True),
    ("pool_stride", 100 * 512 - 16, False), ("page_stride", 500, False), ("page_stride", 256, False), ("page_bytes", 8, False),
    ("page_bytes", 24, False), ("page_bytes", 0, False), ("n_pages", 0, False), ("n_pages", 1 << 25, False),
])
def test_pages_copy(B, cfg, field, value, fine):
    a = B.make_pages_copy_args(5, copies=FAKE, pools=FAKE, n_pools=3, pool_stride=100 * 512, page_stride=512, page_bytes=512,
                               n_pages=100)
    assert B.pages_copy_check(cfg, a) == B.SV_OK
    setattr(a, field, value)
    assert (B.pages_copy_check(cfg, a) == B.SV_OK) == fine


def append_args(B, **more):
    d = dict(cache=cache(B, page_counts=None, page_refs=None, free_pages=None), kv=kv(B), keys=FAKE, values=FAKE,
             strides=(1000, 128, 64))
    d.update(more)
    return B.make_append_args(4, 5, **d)


@pytest.mark.parametrize("field,value", [
    ("B", -1), ("B", 9), ("rows", 0), ("rows", (1 << 20) + 1), ("row0", -1), ("keys", None), ("values", None),
    ("row_stride", 63), ("head_stride", 63), ("batch_stride", -1)])
def test_append_refuses(B, cfg, field, value):
    a = append_args(B)
    assert B.append_check(cfg, a) == B.SV_OK
    setattr(a, field, value)
    assert refused(B.append_check(cfg, a), B)


@pytest.mark.parametrize("more", BAD_CACHES)
def test_append_and_attend_refuse_caches(B, cfg, more):
    assert refused(B.append_check(cfg, append_args(B, cache=cache(B, **more))), B)
    assert refused(B.attend_check(cfg, attend_args(B, cache=cache(B, **more))), B)


@pytest.mark.parametrize("more", BAD_KVS)
def test_append_and_attend_refuse_kvs(B, cfg, more):
    assert refused(B.append_check(cfg, append_args(B, kv=kv(B, **more))), B)
    assert refused(B.attend_check(cfg, attend_args(B, kv=kv(B, **more))), B)


def test_packed_rows_have_no_last_row(B, cfg):
    assert B.append_check(cfg, append_args(B, row_offsets=FAKE, last_row=FAKE)) == B.SV_EINVAL
    assert B.attend_check(cfg, attend_args(B, row_offsets=FAKE, last_row=FAKE)) == B.SV_EINVAL
    assert B.attend_check(cfg, attend_args(B, row_offsets=FAKE)) == B.SV_OK


def attend_args(B, **more):
    d = dict(cache=cache(B, page_counts=None, page_refs=None, free_pages=None), kv=kv(B), heads=8, queries=FAKE,
             query_strides=(2560, 512, 64), outputs=FAKE, output_strides=(2560, 512, 64), scale=0.125, workspace=FAKE,
             workspace_bytes=1 << 40)
    d.update(more)
    return B.make_attend_args(4, 5, **d)


@pytest.mark.parametrize("field,value", [
    ("B", -1), ("B", 9), ("rows", 0), ("rows", 10), ("row0", -1), ("row0", 5), ("heads", 0), ("heads", 7), ("heads", 130),
    ("queries", None), ("outputs", None), ("query_row_stride", 63), ("query_head_stride", 63), ("output_row_stride", 63),
    ("output_head_stride", 63), ("query_batch_stride", -1), ("output_batch_stride", -1), ("scale", float("nan")),
    ("scale", float("inf")), ("window", -1), ("max_len", -1), ("max_len", (1 << 30) + 1), ("workspace", None),
    ("workspace", FAKE + 8), ("workspace_bytes", 15)])
def test_attend_refuses(B, cfg, field, value):
    a = attend_args(B)
    assert B.attend_check(cfg, a) == B.SV_OK
    setattr(a, field, value)
    assert refused(B.attend_check(cfg, a), B)


def test_attend_workspace(B, cfg):
    a = attend_args(B, workspace=None, workspace_bytes=0)
    n = B.attend_workspace_bytes(cfg, a)
    assert n > 0 and n % 16 == 0
    a.workspace, a.workspace_bytes = FAKE, n
    assert B.attend_check(cfg, a) == B.SV_OK
    a.workspace_bytes = n - 1
    assert B.attend_check(cfg, a) == B.SV_EINVAL
    a.max_len = 100  # one tile for each wavefront: not split
    assert B.attend_workspace_bytes(cfg, a) == 0
    a.workspace = None
    assert B.attend_check(cfg, a) == B.SV_OK
    a.heads = 7
    with pytest.raises(B.SpecVerifyError):
        B.attend_workspace_bytes(cfg, a)


def test_attend_refuses_more_rows_of_all_heads_than_a_launch_takes(B):
    cfg = B.Config(8, 256, 100, B.SV_BF16, 0)
    a = attend_args(B, kv=kv(B, kv_heads=1024, head_dim=64, strides=(1 << 20, 1 << 10, 64)), heads=65536, query_strides=(1 << 30, 1 << 22, 64),
                    output_strides=(1 << 30, 1 << 22, 64), workspace_bytes=1 << 60)
    for rows, rc in ((128, B.SV_OK), (129, B.SV_EUNSUPPORTED)):
        a.rows = rows
        assert B.attend_check(cfg, a) == rc


def test_attend_plan(tmp_path):
    """Every row and every token has its workgroup, and the kernels that the plan names exist."""
    src = tmp_path / "plan.cpp"
    src.write_text('''
#include "sv_attend_plan.h"
#include <cstdio>
#include <initializer_list>
int main()
{
    const int dims[] = {64, 128, 256};
    bool used[3][2][10] = {};
    for (int d = 0; d < 3; ++d)
        for (long long rows = 1; rows < 17000; rows += rows < 400 ? 1 : 37)
            for (long long len : {1ll, 127ll, 128ll, 129ll, 4000ll, 131000ll, 1ll << 30})
                for (long long B : {1ll, 3ll, 300ll, 5000ll, 1000000ll})
                    for (int kv : {1, 5, 16, 1024}) {
                        const sv::AttendPlan p = sv::attend_plan(B, kv, dims[d], rows % 2, rows, len);
                        if ((long long)p.blocks * p.rows < rows || p.blocks < 1 || p.rows != p.tiles * (p.shared ? 64 : 16)) return printf("rows %lld\\n", rows), 1;
                        if (p.batch < 1 || p.batch > B || p.batch > 256 || p.shares < 8 || p.shares % 8) return printf("B %lld\\n", B), 1;
                        // the units of a launch, and what is rounded up, stay within 32 bits, and so do its work-items
                        if (p.batch * (sv::attend_units(len) + p.begin) + p.shares > 0x7fffffffll) return printf("len %lld\\n", len), 1;
                        if ((long long)p.shares * kv * p.blocks * 256 > 0xffffffffll) return printf("groups %d %d %d\\n", p.shares, kv, p.blocks), 1;
                        used[d][rows % 2][p.tiles + 4 * p.shared] = true;
                    }
    for (int d = 0; d < 6; ++d) {
        for (int t = 1; t < 10; ++t) if (used[d / 2][d % 2][t]) printf(t > 4 ? "s%d " : "%d ", t > 4 ? t - 4 : t);
        printf("| ");
    }
}
''')
    exe = tmp_path / "plan"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "draft_verification_amd", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert r.stdout.strip() == "1 s1 s2 s3 | 1 2 s1 s2 s3 | 1 2 s1 s2 s3 | 1 2 3 s1 s2 s3 | 1 s1 | 1 s1 |"
