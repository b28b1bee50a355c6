// How the launches of the short convolution (causal_conv.cu) cut up sequences and channels.  Plain C++, so that
// the counts are checked without a GPU up to the largest sizes that a call may have: tokens within 8192 of 2^31, channels
// and sequences up to 2^31 - 1 between them, whose sums pass 31 bits.
#pragma once

#ifdef __CUDACC__
#define TTM_CONV_PLAN __host__ __device__ inline
#else
#define TTM_CONV_PLAN inline
#endif

namespace ttm {

constexpr int kConvSms = 152;
constexpr int kConvThreads = 128;
constexpr int kConvBatch = 4;           // rows whose loads are in flight together

// End of the strip that starts at t0 < T (t0 + strip may be past 2^31).
TTM_CONV_PLAN int conv_strip_end(int T, int t0, int strip) { return strip < T - t0 ? t0 + strip : T; }

inline int conv_strips(int T, int strip) { return (int)(((long long)T + strip - 1) / strip); }

struct ConvFwdPlan {
    int strip, strips;                  // tokens of a strip; strips of a sequence
    long long blocks;
};

// Strips as long as leave two waves of threads, 8 to 128 tokens (the rows between strips are read twice), or one strip.
inline ConvFwdPlan conv_fwd_plan(int N, int T, int groups, bool one_strip) {
    ConvFwdPlan p;
    p.strip = one_strip ? T : 128;
    while (!one_strip && p.strip > 8 && (long long)N * groups * conv_strips(T, p.strip) < kConvSms * 2048LL) p.strip /= 2;
    p.strips = conv_strips(T, p.strip);
    p.blocks = ((long long)N * groups * p.strips + kConvThreads - 1) / kConvThreads;
    return p;
}

// Rows of the gradient's grid at most, one wave by the widest channel groups that a call may take; the workspace
// holds a part for each.
inline int conv_most_rows(int C) {
    const long long across = (((long long)C + 3) / 4 + 31) / 32;
    const int rows = (int)(kConvSms * 4 / across);
    return rows < 1 ? 1 : rows;
}

struct ConvBwdPlan {
    int bx, by;                         // threads of a block: channel groups, strips
    int across, rows;                   // the grid: blocks of channel groups, rows of strips
    int strip, strips;
};

// One strip a thread where the sequences are fewer than the threads of a column of the grid, of 16 tokens at least.
inline ConvBwdPlan conv_bwd_plan(int N, int T, int C, int groups, int blocks_per_sm) {
    ConvBwdPlan p;
    p.bx = 1;
    while (p.bx < groups && p.bx < 32) p.bx *= 2;
    p.by = kConvThreads / p.bx;
    p.across = (int)(((long long)groups + p.bx - 1) / p.bx);
    p.rows = kConvSms * blocks_per_sm / p.across;
    if (p.rows > conv_most_rows(C)) p.rows = conv_most_rows(C);
    if (p.rows < 1) p.rows = 1;
    const long long places = (long long)p.rows * p.by, each = places / N;
    const long long strip = each <= 1 ? T : ((long long)T + each - 1) / each;
    p.strip = strip < 16 ? 16 : (int)((strip + kConvBatch - 1) / kConvBatch * kConvBatch);
    p.strips = conv_strips(T, p.strip);
    const long long wanted = ((long long)N * p.strips + p.by - 1) / p.by;
    if (wanted < p.rows) p.rows = (int)wanted;
    return p;
}

}  // namespace ttm

#undef TTM_CONV_PLAN
