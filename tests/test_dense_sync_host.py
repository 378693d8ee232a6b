"""The two-SM kernel's synchronisation, from its source: what one SM of a pair, or
an asynchronous engine, sends to the other's barriers is waited for there before
the pair leaves."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KERNEL = open(os.path.join(ROOT, "nvfp4_weight_only_router_b200", "csrc", "dense", "pair_gemm.cu")).read()


def _between(start, end):
    i = KERNEL.index(start)
    return KERNEL[i:KERNEL.index(end, i)]


def test_last_arrivals_are_waited_for():
    # commits of a stage's products arrive on `empty` in both SMs: the producer that
    # both SMs have drains every stage behind its loop
    tail = _between("sm.issued[turn] = issued", "} else if (warp == kPMma)")
    assert re.search(r"for \(int i = 0; i < C::NS && ok; \+\+i\) \{\s*ok = swait\(sm, &sm\.empty\[s\], parity", tail)
    # the epilogues of both SMs arrive on SM 0's `d_empty`: the issuer waits for the
    # last use of each accumulator; the final commit arrives in both, which both wait for
    end = _between("commit_pair(&sm.fin)", "warp == kPScale")
    assert "pwait(sm, &sm.d_empty[db], ((titer - 1 - db) >> 1) & 1" in end
    leader, both = end.split("    }\n    mbar_wait_bounded(&sm.fin, 0);")
    assert "d_empty" in leader and "mbar_wait_bounded" not in leader and "__syncwarp" in both


def test_parity_of_the_last_use():
    """The issuer's formula against the barrier's phases: use k (from 0) of an
    accumulator completes the phase of parity k & 1."""
    for tiles in range(1, 40):
        for db in range(2):
            uses = len([t for t in range(tiles) if t % 2 == db])
            assert (uses > 0) == (tiles > db)
            if uses:
                assert ((tiles - 1 - db) >> 1) & 1 == (uses - 1) & 1


def test_every_stage_is_drained_once():
    """The producer's closing waits from its state (s, parity): each stage's last
    phase, or the one before a stage's first use, which a fresh barrier passes."""
    for ns in (3, 4, 7):
        for issued in range(0, 5 * ns):
            s, parity = issued % ns, 1 ^ ((issued // ns) & 1)
            seen = set()
            for _ in range(ns):
                uses = len(range(s, issued, ns))           # of stage s
                # waiting for parity q passes once the phase of index k with k & 1 == q is the
                # last completed one (k = uses - 1; -1 on a fresh barrier)
                assert parity == (uses - 1) & 1
                seen.add(s)
                s += 1
                if s == ns:
                    s, parity = 0, parity ^ 1
            assert len(seen) == ns


def test_remote_arrivals_name_their_scope():
    """An arrival on the other SM's barrier without a scope is ordered for its own
    block alone.  Converters publish shared memory: a cluster-wide release, and the
    issuer's wait acquires at that scope."""
    forms = re.findall(r"mbarrier\.arrive\.[\w.:]*shared::cluster\.b64", KERNEL)
    assert sorted(set(forms)) == ["mbarrier.arrive.relaxed.cluster.shared::cluster.b64",
                                  "mbarrier.arrive.release.cluster.shared::cluster.b64"]
    convert = _between("auto convert = ", "Stage even, odd;")
    assert "arrive_written(full0" in convert and "arrive_read" not in convert
    assert "mbarrier.arrive.release" in _between("void arrive_written", "\n}")
    issue = _between("MMA issuer", "every MMA issued has completed")
    assert "if constexpr (KIND == kKindW4) ok = swait_written(sm, &sm.full[s]" in issue
    assert "mbarrier.try_wait.parity.acquire.cluster" in _between("bool try_wait_cluster", "\n}")


def test_the_next_kernel_starts_behind_the_wait():
    """let_next() directly follows after_previous() in every kernel: a kernel that waits
    for its predecessor knows everything before that one complete as well."""
    import glob
    found = 0
    for path in glob.glob(os.path.join(ROOT, "nvfp4_weight_only_router_b200", "csrc", "dense", "*.cu")):
        src = open(path).read()
        for call in re.finditer(r"\blet_next\(\);", src):
            assert re.search(r"after_previous\(\);\s*$", src[:call.start()]), (path, src[call.start() - 80:call.end()])
            found += 1
        assert len(re.findall(r"\bafter_previous\(\);", src)) == len(re.findall(r"\blet_next\(\);", src)), path
    assert found >= 7
