// How the launches of the short convolution (causal_conv.cu) cut up sequences and channels.  Plain C++, so that
// the counts are checked without a GPU up to the largest sizes that a call may have: tokens within 8192 of 2^31,
// where the sum of two sizes passes 31 bits.
#pragma once

namespace ttm {

constexpr int kConvSms = 152;
constexpr int kConvThreads = 128;
constexpr int kConvBatch = 4;           // rows whose loads are in flight together

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

}  // namespace ttm
