// The scoring and top-k workspace.  Plain C++: no CUDA header is needed to lay it out.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace dsa {

constexpr int kHistBits = 11;
constexpr int kHistBins = 1 << kHistBits;
constexpr int kCandCap = 8192;        // level-1 candidates kept per split row
constexpr int kMaxScoreCtas = 1024;   // largest scoring grid the plan table holds

// Byte offsets of the regions of a dsa_score_paged / dsa_topk workspace.
// Every region starts on a 256-byte boundary.
struct WsLayout {
    size_t hist;        // uint32[rows][2048]: histogram of the top 11 order-preserving score bits
    size_t counters;    // int[rows][4]: winners published, candidates published, spans done, candidates dropped
    size_t zeroed;      // bytes of these two, from the workspace's start
    size_t info;        // int[8]: segment count, tile count
    size_t segs;        // int4[rows + 1]: request, first row, rows, largest bound
    size_t seg_prefix;  // int[rows + 2]: exclusive prefix of tiles per segment
    size_t eff_end;     // int[rows]: row bounds after validation (0 outside every request)
    size_t cta;         // int4[kMaxScoreCtas]: per scoring CTA {first tile, end tile, first segment, segments}
    size_t cand;        // uint2[rows][kCandCap]: level-1 candidates of split rows (key, position)
    size_t logits;      // float[rows][width] when the caller keeps no logits
    size_t total;
};

// The layout in a workspace of `bytes` (0: one just large enough).  The
// histograms and counters must be zero on entry and are zero again when a call
// completes; they lie at the start.  What a call leaves behind lies at the end:
// so calls of different sizes may follow each other in one workspace, none larger
// in rows or width than it was sized for, and none finds another's leavings where
// it counts.
inline WsLayout workspace_layout(int64_t rows, int64_t width, bool with_plan, bool with_logits, size_t bytes = 0) {
    WsLayout L{};
    const size_t r = static_cast<size_t>(rows);
    size_t off = 0;
    auto take = [&](size_t n) {
        const size_t at = off;
        off = (off + n + 255) & ~size_t(255);
        return at;
    };
    L.hist = take(r * kHistBins * 4);
    L.counters = take(r * 4 * 4);
    L.zeroed = off;
    L.info = take(with_plan ? 8 * 4 : 0);
    L.segs = take(with_plan ? (r + 1) * 16 : 0);
    L.seg_prefix = take(with_plan ? (r + 2) * 4 : 0);
    L.eff_end = take(with_plan ? r * 4 : 0);
    L.cta = take(with_plan ? kMaxScoreCtas * 16 : 0);
    L.cand = take(r * kCandCap * 8);
    L.logits = take(with_logits ? r * static_cast<size_t>(width) * 4 : 0);
    L.total = off;
    if (bytes > L.total) {
        const size_t up = (bytes - L.total) & ~size_t(255);
        for (size_t* at : {&L.info, &L.segs, &L.seg_prefix, &L.eff_end, &L.cta, &L.cand, &L.logits}) *at += up;
    }
    return L;
}

}  // namespace dsa
