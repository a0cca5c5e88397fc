"""What the linear-attention kernels share, from their header, compiled for the host.
How packed sequences are cut into items: every token of every sequence is in one item, numbers and
slots never meet, and all of them lie inside the grid and the workspace, also for
offsets that break the rules."""
from __future__ import annotations

import os
import subprocess

import pytest

from ssd_chunked_forward_b200 import ssd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ssd_chunked_forward_b200", "csrc")

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>
#include "linear.h"
using namespace ssd;
static int clamp(int x, int T) { return x < 0 ? 0 : x > T ? T : x; }
static void need(bool ok, const char* what, int line) {
    if (!ok) { std::printf("%s (line %d)\n", what, line); std::exit(1); }
}
#define NEED(x) need(x, #x, __LINE__)

static void run(const std::vector<int>& cu, int T, int seg, int H, int roles, bool valid) {
    ScanPlan p = {};
    p.B = (int)cu.size() - 1; p.T = T; p.H = H; p.nroles = roles; p.packed = 1; p.seg_tokens = seg;
    p.items = ((long long)p.B + T / seg) * H * roles;
    const int HR = H * roles;
    std::set<long long> slots;
    const unsigned whole = T / seg;
    // what the warps' search finds: the last sequence whose first number is at most this one
    auto rows = [&](int s, int& a, int& b) { a = clamp(cu[s], T); b = std::max(a, clamp(cu[s + 1], T)); };
    auto item = [&](long long it) {
        ScanItem r; r.valid = 0; r.slot = r.slot_prev = r.slot_init = -1;
        const unsigned number = (unsigned)(it / HR);
        int a = 0, b = 0, s = -1;
        if (number < whole) {
            for (int i = 0; i < p.B; ++i)
                if ((unsigned)clamp(cu[i], T) / seg <= number) s = i;
        } else s = (int)(number - whole);
        if (s >= 0) { rows(s, a, b); packed_item(p, number, (int)(it % HR), s, a, b, r); }
        return r;
    };
    std::vector<std::set<long long>> seen(p.B), states(p.B);
    long long most = p.slots();
    for (long long it = 0; it < p.items; ++it) {
        ScanItem r = item(it);
        if (!r.valid) continue;
        for (int rev = 0; rev < 2; ++rev) {
            scan_item_tokens(r, seg, rev);
            NEED(r.t0 >= 0 && r.t0 <= r.t1 && r.t1 <= r.len && r.row0 >= 0 && r.row0 + r.len <= T);
            NEED(r.t1 - r.t0 <= seg || r.nseg == 1);
        }
        NEED(r.head >= 0 && r.head < H && r.role >= 0 && r.role < roles && r.seg >= 0 && r.seg < r.nseg);
        if (r.nseg > 1) {
            NEED(r.slot_init >= 0 && r.slot_init < most && r.slot_prev >= 0 && r.slot_prev < most);
            NEED(p.cut());
        } else NEED(r.slot_prev == -1);
        NEED(seen[r.seq].insert((long long)r.seg * HR + r.head * roles + r.role).second);
    }
    for (long long it = 0; p.cut() && it < p.state_items(); ++it) {
        ScanItem r = item(it);
        if (!r.valid || r.seg == r.nseg - 1) continue;
        NEED(r.slot >= 0 && r.slot < most && r.slot_init < most);
        if (!valid) continue;
        NEED(slots.insert(r.slot).second);
        if (r.seg == 0) NEED(slots.insert(r.slot_init).second);
        NEED(states[r.seq].insert((long long)r.seg * HR + r.head * roles + r.role).second);
    }
    if (!valid) {  // whichever sequence a search finds
        for (long long it = 0; it < p.items; ++it)
            for (int s = 0; s < p.B; ++s) {
                const unsigned number = (unsigned)(it / HR);
                int a, b;
                rows(s, a, b);
                if (number < whole ? (unsigned)a / seg > number : (int)(number - whole) != s) continue;
                ScanItem r; r.slot = r.slot_prev = r.slot_init = -1;
                packed_item(p, number, (int)(it % HR), s, a, b, r);
                if (!r.valid) continue;
                scan_item_tokens(r, seg, 0);
                NEED(r.seg >= 0 && r.t0 >= 0 && r.t1 <= r.len && r.row0 + r.len <= T);
                if (r.nseg > 1) NEED(r.slot_prev >= 0 && r.slot_prev < most && r.slot_init < most);
                if (it < p.state_items() && r.seg < r.nseg - 1) NEED(r.slot >= 0 && r.slot < most);
            }
        return;
    }
    for (int s = 0; s < p.B; ++s) {
        const int len = cu[s + 1] - cu[s], n = len <= seg ? 1 : (len + seg - 1) / seg;
        NEED((int)seen[s].size() == n * HR);
        NEED((int)states[s].size() == (n - 1) * HR);
    }
    if (p.cut()) NEED(most <= 2LL * (T / seg) * HR);
}

// the last item of a sequence whose length is the largest that a call takes
static void longest(int seg, int packed) {
    ScanPlan p = {};
    p.B = 1; p.T = 0x7fffffff - 1024; p.H = p.nroles = 1; p.packed = packed; p.seg_tokens = seg;
    const int n = (p.T - 1) / seg + 1;
    long long tokens = 0;
    for (int i = 0; i < n; ++i) {
        ScanItem r; r.slot = r.slot_prev = r.slot_init = -1;
        if (packed) packed_item(p, (unsigned)i, 0, 0, 0, p.T, r);
        else r.len = p.T, r.seg = i, r.nseg = n;
        NEED(r.nseg == n);
        scan_item_tokens(r, seg, i & 1);
        NEED(r.t0 >= 0 && r.t0 < r.t1 && r.t1 <= p.T);
        scan_item_tokens(r, seg, 0);
        tokens += r.t1 - r.t0;
    }
    NEED(tokens == p.T);
}

// blocks on CUDA cores: eight neighbouring rows' 16-byte reads meet 32 different banks,
// and every size fits
static void layouts() {
    for (int K = 1; K <= 256; ++K) {
        const SimtLayout l = simt_layout(K);
        std::set<int> banks;
        for (int row = 0; row < 8; ++row)
            for (int word = 0; word < 4; ++word) banks.insert((row * l.ldk + word) % 32);
        NEED(banks.size() == 32 && l.ldk >= l.K4 && l.K4 >= K && l.ldk % 4 == 0);
        NEED(l.bytes <= simt_layout(256).bytes && l.bytes <= 226 * 1024);
    }
}

int main() {
    layouts();
    for (int packed = 0; packed < 2; ++packed) {
        longest(1 << 30, packed);
        longest(4836224, packed);
        longest(512, packed);
    }
    std::srand(7);
    for (int round = 0; round < 4000; ++round) {
        const int B = 1 + std::rand() % 40, T = 1 + std::rand() % 3000, seg = 1 + std::rand() % 400;
        std::vector<int> cu(B + 1);
        const bool valid = round % 3 != 0;
        if (valid) {  // gaps before and behind, empty ones, one long one among many short
            int left = T, at = std::rand() % (T + 1);
            for (int i = 0; i <= B; ++i) {
                cu[i] = at;
                left = T - at;
                at += std::rand() % 3 == 0 ? 0 : std::rand() % (std::rand() % 4 == 0 ? left + 1 : left / B + 1);
            }
        } else {
            for (int i = 0; i <= B; ++i) cu[i] = std::rand() % (2 * T) - T / 2;
        }
        run(cu, T, seg, 1 + std::rand() % 3, 1 + std::rand() % 3, valid);
    }
    std::puts("ok");
}
"""


def test_items_and_layouts(tmp_path):
    src, exe = tmp_path / "items.cpp", tmp_path / "items"
    src.write_text(PROGRAM)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    res = subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.join(cuda, "include"), str(src), "-o",
                          str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stdout


@pytest.mark.parametrize("B,T,H", [(1000, 100000, 32), (4096, 65536, 32), (24, 18011, 16), (1, 1 << 20, 2)])
def test_workspace_does_not_grow_with_the_sequences(B, T, H):
    """Slots are the cut sequences': at most two for every cut distance of the rows, a
    distance being about three items for every one that runs at a time."""
    from ssd_chunked_forward_b200.build import build
    build()
    K = V = 128
    shape = ssd.LinearShape(B, T, H, H, K, V, ssd.SSD_DTYPE_BF16, 1)
    one = ssd.LinearShape(1, T, H, H, K, V, ssd.SSD_DTYPE_BF16, 1)
    for size, chains in ((ssd.linear_workspace_size, H), (ssd.linear_backward_workspace_size, 3 * H)):
        assert size(shape) == size(one)
        # distances: three items for each of 148 blocks, rounded to whole chunks (a third more at most)
        assert size(shape) <= 256 + 256 + 2 * (4 * 148 + chains) * K * V * 4
