// la_delta_plan.h -- which way la_delta_extend takes a batch by chunks: whole chains, segments of long ones
// side by side, or segments planned on the device.  Rules on sizes alone, free of CUDA, so that a plain
// C++ program can try them for any number of SMs.
#pragma once

#ifdef __CUDACC__
#define LA_HD __host__ __device__
#else
#define LA_HD
#endif

namespace la {

constexpr int kDeltaChunk = 64;  // tokens of a chunk

// A chain cut into segs segments, the first ratio times as long as the others; segs == 1: whole.
struct Cut {
    int segs, ratio;
};
constexpr int kMaxSegs = 32;
constexpr int kSplitSMs = 152;       // SMs of a GB300: chains that run side by side (fewer SMs: the same, in waves)
constexpr int kSplitMinChunks = 20;  // shorter requests are not split
// What the join and two more launches cost, and a segment in the join, in chunks of the chain.
constexpr double kSplitCost = 5., kJoinCost = 1.;
constexpr double kSplitGain = .95;  // a split has to promise this much
// Chunks of segments 1, 2 ..; the last segment that has any.  A short request beside long ones (or under a
// max_seqlen that none comes near) stays whole.
LA_HD inline int split_base(const Cut &s, int nchunks) {
    if (nchunks < kSplitMinChunks) return nchunks;
    return (nchunks + s.ratio + s.segs - 2) / (s.ratio + s.segs - 1);
}
LA_HD inline int split_last(const Cut &s, int nchunks) {
    const int base = split_base(s, nchunks), rest = nchunks - s.ratio * base;
    return rest > 0 ? 1 + (rest - 1) / base : 0;
}
// Matrices of a split: at most two per chain that runs in pass 2, (segs - 1) chains <= kSplitSMs.
inline unsigned long long split_mats(long long chains, long long chunks) {
    if (chunks < kSplitMinChunks || 2 * chains > kSplitSMs) return 0ull;
    const long long most = chains * (2 * kMaxSegs - 3);
    return (unsigned long long)(most < 2 * kSplitSMs ? most : 2 * kSplitSMs);
}
// The split whose longest way through both passes is shortest, in chunks: a pass 1 with ratio of the
// short chains one after another beside a segment 0, then a segment of pass 2, and what the join and its
// launches cost.
inline Cut plan_split(long long chains, long long chunks) {
    Cut s{1, 1};
    if (split_mats(chains, chunks) == 0) return s;
    double best = kSplitGain * (double)chunks;
    for (int ratio = 1; ratio <= 2; ++ratio)
        for (int segs = 3; segs <= kMaxSegs && (segs - 1) * chains <= kSplitSMs; ++segs) {
            if (2 * (segs - 2) * chains > ratio * (kSplitSMs - chains)) continue;
            const Cut t{segs, ratio};
            const double cost = (ratio + 1) * split_base(t, (int)chunks) + kSplitCost + kJoinCost * segs;
            if (cost < best) {
                best = cost;
                s = t;
            }
        }
    return s;
}

// Requests: planning is a pass over all of them per pair of lengths tried, which 512 short ones made 50 us
// longer than T takes.
constexpr int kMaxPlanned = 128;
// Longest request: one of 1500 tokens among 127 of 64, 4 heads, takes 83 us with a plan and 76 without; of 2000
// 78 and 93.
constexpr int kPlanMinChunks = 32;
constexpr int kPlanMats = 512;  // matrices (start states and transitions, all heads)
// Whether a batch gets a plan: more chains than a split takes, and a longest request (of `longest` chunks) of
// at least twice the SMs' even share of all chunks, 8 added to it.  At 16 heads, without / with, us: 16,384
// tokens among 63 x 256: 707 / 426; 8192, 4096, 6 x 500: 352 / 227; 4096 among 7 x 1024 (2.4 times): 193 / 169,
// among 7 x 1536 (2.0): 204 / 201; eight of 512-4096 (1.7): 218 / 212 and 218 / 229; twelve of 256-4096 (1.1):
// 221 / 232.
inline bool planned(long long B, long long H, long long chunks, long long longest) {
    return 2 * B * H > kSplitSMs && B >= 2 && B <= kMaxPlanned && H <= kPlanMats && longest >= kPlanMinChunks &&
           longest * kSplitSMs >= 2 * (H * chunks + 8 * kSplitSMs);
}

constexpr int kMaxRanked = 8192;  // requests of a batch that is taken longest first

// How a batch of T > 0 tokens runs on num_sms SMs.
struct Schedule {
    bool planned;  // as segments planned on the device
    Cut cut;       // otherwise: the cut of its chains
    bool ranked;   // whole chains, longest first
};
inline Schedule make_schedule(long long B, long long T, long long H, long long max_seqlen, int num_sms) {
    const long long chunks = (T + kDeltaChunk - 1) / kDeltaChunk;
    const long long longest = ((max_seqlen < T ? max_seqlen : T) + kDeltaChunk - 1) / kDeltaChunk;
    Schedule s{planned(B, H, chunks, longest), {1, 1}, false};
    if (s.planned) return s;
    s.cut = plan_split(B * H, longest);
    // One wave needs no order; ranking is B comparisons per request.  A split's chains keep the order of the
    // batch, by which the join finds them, and have a CTA each: where fewer SMs than chains are visible (the
    // split's rule counts kSplitSMs of them) they run in waves.
    s.ranked = s.cut.segs == 1 && B > 1 && B <= kMaxRanked && B * H > num_sms;
    return s;
}

}  // namespace la
