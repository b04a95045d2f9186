// Layer norm's launch shapes: how many warps hold a row, how many such groups a CTA has, and how rows are staged in shared memory.
// Plain C++, so that the limits that the kernels rely on can be checked for every width without a GPU.
#pragma once

namespace mhc {

constexpr int kLnThreads = 512;                     // of a CTA: as many groups as fit
constexpr int kLnMaxHeld = 8192;                    // columns that a group holds in registers
constexpr int kLnArrays = 3;                        // that are staged
constexpr int kLnMostStages = 4;
constexpr int kLnAllBarrier = 15;                   // named barrier of all groups; a group of several warps has its number + 1

inline int ln_runs8(int H) { return (H + 255) / 256; }      // warps of one run of 8 columns a lane
inline int ln_up(int v, int to) { return (v + to - 1) / to * to; }
inline int ln_least(int a, int b) { return a < b ? a : b; }

// A stage's places for rows of these sizes (0: none), wherever the rows begin, and its size; a run read past a row's end
// touches at most 48 bytes more.
inline void ln_places(const int (&row_bytes)[kLnArrays], int (&place)[kLnArrays + 1]) {
    int at = 0;
    for (int i = 0; i < kLnArrays; ++i) {
        place[i] = at;
        if (row_bytes[i]) at += ln_up(row_bytes[i] + 15 + 64, 128);
    }
    place[kLnArrays] = at;
}

// Forward, rows from memory to registers: groups of `warps` warps, R runs of 8 columns a thread.
struct LnRows {
    int R, warps, groups;
};
inline LnRows ln_rows(int H) {
    LnRows s;
    const int need = ln_runs8(H);
    s.R = need <= 1 ? 1 : need <= 2 ? 2 : 4;
    s.warps = (need + s.R - 1) / s.R;
    s.groups = kLnThreads / (32 * s.warps);
    return s;
}

// Forward, staged rows: a CTA an SM, as many groups as 768 threads give beside the warp that orders rows, as many stages as shared memory
// holds. Barriers, the parameters in fp32, then the groups' stages.
constexpr int kLnRingThreads = 768, kLnRingSmem = 220 * 1024, kLnRingBars = 512, kLnRingGroups = 8;
struct LnRingShape {
    int R, warps, groups, stages, params, smem;
};
inline LnRingShape ln_ring_shape(int H, int stage_bytes, bool runs, bool affine) {
    LnRingShape s;
    // four runs a thread leave too few registers for rows that are shifted into place; others take four from 1537 columns on (8192 rows of bf16:
    // 4096 columns 31 us against 36 with two, 7168 52 against 70, but 2048 17.6 against 17.5 and 1024 12.0 against 11.3)
    const int need = ln_runs8(H);
    s.R = need <= 6 || !runs ? 2 : 4;
    s.warps = (need + s.R - 1) / s.R;
    s.groups = ln_least((kLnRingThreads - 32) / (32 * s.warps), kLnRingGroups);
    s.params = affine ? ln_up(8 * ln_up(H, 8), 128) : 0;
    s.stages = ln_least((kLnRingSmem - kLnRingBars - s.params) / (s.groups * stage_bytes), kLnMostStages);
    s.smem = kLnRingBars + s.params + s.groups * s.stages * stage_bytes;
    return s;
}

// Backward: as many groups as 512 threads give, a CTA an SM of `sms`. With several rows a group they are staged, by one more
// warp, or (self) by each group's first thread where that warp would cost a group. parts: CTAs. Staged against from memory, with
// d_residual, among rows that L2 does not hold: 8192 x 4096 bf16 52 us against 98, 8192 x 520 16.5 against 21.3, 2432 x 2048 15.2 against 19.1, 2432 x 1024
// 11.4 against 11.9; a row a group: 608 x 2048 10.2 against 9.1, 1216 x 1024 9.9 against 8.5. Up to 256 columns a thread holds one run, and a CTA 16 rows.
constexpr int kLnBackRuns = 2, kLnBackRingSmem = 216 * 1024, kLnBackRingBars = 1024;
constexpr int kLnBackMeetSmem = 64 * 1024;          // 512 threads of two runs: 8192 columns in all groups, two sums
struct LnBack {
    int R, warps, groups, parts;
    bool ring, self;
};
inline LnBack ln_back(long long T, int H, int sms) {
    LnBack p = {1, kLnThreads / 32, 1, 0, false, false};
    if (H <= kLnMaxHeld) {
        const int need = ln_runs8(H);
        p.R = need <= 1 ? 1 : kLnBackRuns;
        p.warps = (need + p.R - 1) / p.R;
        p.groups = kLnThreads / (32 * p.warps);
        if (p.R == kLnBackRuns && T > static_cast<long long>(sms) * p.groups) {
            p.ring = true;
            p.self = p.warps % 8 == 0;
            if (!p.self) p.groups = (kLnThreads - 32) / (32 * p.warps);
        }
    }
    const long long blocks = (T + p.groups - 1) / p.groups;
    p.parts = static_cast<int>(blocks < sms ? blocks : sms);
    return p;
}
inline int ln_back_meet(const LnBack &p, int H) { return p.groups * 8 * ln_up(H, 8); }      // bytes in which the groups' sums meet
// The staged form's: barriers, the weight in fp32, then the stages, or what meets in them. stages: none where it cannot run (with
// d_residual a group's first thread orders a row later: two places at least).
struct LnBackRing {
    int stages, params, smem;
};
inline LnBackRing ln_back_ring(const LnBack &p, int H, int stage_bytes, bool residual) {
    LnBackRing s;
    s.params = ln_up(4 * ln_up(H, 8), 128);
    s.stages = ln_least((kLnBackRingSmem - kLnBackRingBars - s.params) / (p.groups * stage_bytes), kLnMostStages);
    if (s.stages < (p.self && residual ? 2 : 1)) s.stages = 0;
    const int places = p.groups * s.stages * stage_bytes, meet = ln_back_meet(p, H);
    s.smem = kLnBackRingBars + s.params + (places > meet ? places : meet);
    return s;
}

}  // namespace mhc
