// route_grouped.cu -- from router logits to top-k ids, weights, counts and the
// balance loss, with softmax or sigmoid scores, a bias that takes part in the
// choice alone, and groups of experts of which the best few stay.
//
// A warp owns a token and holds its row as route.cu does; the picks, the sums
// and their order are that kernel's too.  What differs is that the choice goes
// by computed values, c = s + bias, where route.cu's goes by the logits
// themselves: fp32 scores are off by a few units in the last place, and two
// experts nearer than that could come out in the wrong order (of 16384 tokens
// with 256 experts some 15 have such a pair).  So every choice is checked
// against a bound on its error, and where that fails the experts in question are
// valued again: in sums of two floats (fixed_key), for they leave one token in
// some 500 of these open again, which is then chosen in 64 bits after the loop
// (settle).  Without a bias, or with one alike for all, the picks go by logits,
// and only the groups' values need the check.  What a rare path costs here is the
// fetching of its instructions, and the call ends with its slowest block: a
// choice in 64 bits of all that was open took 10 to 25 us of a call of 25.
//
// 16384 x 256 fp32, K = 8, bias, the best 4 of 8 groups: 28.6 us; without groups
// and bias 24.3 (moe_route, with softmax: 19.0); some 2 us more where tokens are
// valued again, 10 to 13 where one is left for settle.  No single thing bounds it.
// A multiprocessor has a block in 65 % of the kernel's cycles: some 8 us are the two
// launches, and a warp has 3.37 tokens, so that 37 % of the blocks have a fourth
// round that the others wait for.  In those cycles 62 % of the issue slots are used,
// by 882 instructions a token (724 without groups and bias, moe_route 478); the
// warps wait for one another's slots, for results in a token's chain of dependent
// steps, and for shared and global memory, about as much for each.  32 warps a
// multiprocessor (24: 32.3 us, 16 in larger blocks 30.9) leave 64 registers a
// thread: this form spills 76 bytes of stores and 68 of loads, 1.6 % of its
// instructions.  One token: 4.9 us.
#include "activation.cuh"
#include "route_grouped.cuh"
#include "route_totals.cuh"

#include <cfloat>
#include <limits>

namespace moe {
namespace {

constexpr int kWarps = 8;                            // a block
// Blocks a multiprocessor, by the registers of NV values a lane.
constexpr int per_sm(int NV) { return NV <= 8 ? 4 : NV <= 12 ? 3 : NV <= 16 ? 2 : 1; }
// Words of a lane's sorted list: none where a lane has too many values to sort.
constexpr int list_of(int NV) { return NV <= 16 ? NV + 4 : 0; }
constexpr int kOpen = -2;                            // in a token's first id: chosen after the loop
constexpr float kUnit = 5.9604645e-8f;               // 2^-24

struct Rules {
    const float *bias;                               // [E] or null
    int softmax, groups, top_groups, group_top, renorm;
    float scale;
};

// A value to choose by: NaN is behind every number.
__device__ __forceinline__ float rankable(float c) { return fmaxf(c, -FLT_MAX); }

// The two largest of a warp's pairs a >= b (each lane's), over `lanes` lanes.
__device__ __forceinline__ void top_two(float &a, float &b, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) {
        const float a2 = __shfl_xor_sync(kFullMask, a, o), b2 = __shfl_xor_sync(kFullMask, b, o);
        b = fmaxf(fminf(a, a2), fmaxf(b, b2));
        a = fmaxf(a, a2);
    }
}

template <typename T>
__device__ __forceinline__ void top_two(T &a, T &b, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) {
        const T a2 = __shfl_xor_sync(kFullMask, a, o), b2 = __shfl_xor_sync(kFullMask, b, o);
        const T low = a2 < a ? a2 : a, second = b2 > b ? b2 : b;
        a = a2 > a ? a2 : a;
        b = low > second ? low : second;
    }
}

template <typename T>
__device__ __forceinline__ void insert(T v, T &a, T &b)
{
    if (v > a) {
        b = a;
        a = v;
    } else if (v > b) {
        b = v;
    }
}

// The same with the logit that each value is of.
__device__ __forceinline__ void insert(long long v, float x, long long &a, float &ax, long long &b, float &bx)
{
    if (v > a) {
        b = a;
        bx = ax;
        a = v;
        ax = x;
    } else if (v > b) {
        b = v;
        bx = x;
    }
}

// A group's value from its largest two (-inf: no open expert).  NaN keys hold the
// type's lowest value, and so does a value with one in it: behind every number's,
// before a group without an open expert.  A sum past the type's range is cut there.
template <typename T>
__device__ __forceinline__ T group_value(T a, T b, int group_top)
{
    constexpr T kLast = std::numeric_limits<T>::lowest();
    if (group_top != 2 || !(b > -INFINITY)) return a;
    return b > kLast ? max(min(a + b, -kLast), kLast) : b;
}

// A lane's NV values to and from a row of 32 NV in shared memory.
template <int NV>
__device__ __forceinline__ void store_own(float *row, int lane, const float (&v)[NV])
{
    static_assert(NV % 4 == 0);
#pragma unroll
    for (int j = 0; j < NV; j += 4)
        *reinterpret_cast<float4 *>(row + lane * NV + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
}

template <int NV>
__device__ __forceinline__ void load_own(const float *row, int lane, float (&v)[NV])
{
#pragma unroll
    for (int j = 0; j < NV; j += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(row + lane * NV + j);
        v[j] = q.x;
        v[j + 1] = q.y;
        v[j + 2] = q.z;
        v[j + 3] = q.w;
    }
}

// What a row's scores are made with: softmax's maximum and the reciprocal of its sum.
struct Row {
    float m, inv;
};

__device__ __forceinline__ float score_of(float x, const Rules &r, const Row &row)
{
    return r.softmax ? weight_of(x, row.m) * row.inv : sigmoid_approx(x);
}

// Differences of keys and of group values that fp32 cannot tell from 0.
struct Room {
    float keys, groups;
};

// With u = 2^-24, scores of at most `top` and |c| <= top + largest.  The power of
// 2 is off by (1.22 |z| + 4) u of itself, z its argument's size (the product with
// log2(e) and that number's rounding, and 2 ulp for the power).  That moves a
// logistic score by s (1 - s) times as much: at most 1.3 u, and 112 u top where top
// is small (|z| <= 88); its sum adds u top and the reciprocal one ulp, 2 u top.  A
// softmax score, whose z is a rounded difference, has (2.22 |z| + 4) u of its own,
// |z| top below 0.4; 20 from the sum's terms (their mean |z| is below log 1024),
// 37 additions, 4 from the quotient and 1 from the product: below 70 u top.  The
// sum with the bias adds u (top + largest).  Two keys: twice that; two groups'
// values: four times, and their own sums' roundings.  A tenth is added for the
// products of errors.
__device__ __forceinline__ Room room_of(float top, bool softmax, float largest_bias)
{
    const float c = top + largest_bias;
    const float key = (softmax ? 70.0f * top : top > 0.25f ? 1.3f + 3.0f * top : 115.0f * top) + c;
    return {2.2f * kUnit * key, 4.4f * kUnit * (key + c)};
}

// A number as the sum of two floats, the second below the first one's last place
// (Dekker's and Knuth's sums and products).
struct Two {
    float h, l;
};

__device__ __forceinline__ Two two_sum(float a, float b)
{
    const float h = __fadd_rn(a, b), t = __fsub_rn(h, a);
    return {h, __fadd_rn(__fsub_rn(a, __fsub_rn(h, t)), __fsub_rn(b, t))};
}

__device__ __forceinline__ Two two_product(float a, float b)
{
    const float h = __fmul_rn(a, b);
    return {h, __fmaf_rn(a, b, -h)};
}

// exp(a + b), the sum's size at most 80, to 2^-33 of itself, times 2^-n.  The
// argument less n ln 2 (ln 2 in two parts, the first short enough for exact
// products) is r, below 0.35: 1 + r + r^2 / 2 + r^3 / 6 in two floats, what
// follows, below 2^-10, in one.
__device__ __forceinline__ Two two_exp(float a, float b, int &n)
{
    constexpr float kLn2 = 0.693145751953125f, kLn2Rest = 1.42860682030941723e-6f;       // 15 bits, and the rest
    constexpr float kSixth = 0.16666667163372040f, kSixthRest = -4.967053879e-9f;
    const float k = rintf(__fmul_rn(a, kLog2e));
    n = (int)k;
    Two r = two_sum(__fmaf_rn(-k, kLn2, a), __fsub_rn(b, __fmul_rn(k, kLn2Rest)));
    const float h = r.h;
    const Two square = two_product(h, h);
    Two cube = two_product(square.h, h);
    cube.l = __fmaf_rn(square.l, h, cube.l);
    Two third = two_product(cube.h, kSixth);
    third.l += __fmaf_rn(cube.h, kSixthRest, __fmul_rn(cube.l, kSixth));
    float q = 1.0f / 362880.0f;
    q = __fmaf_rn(q, h, 1.0f / 40320.0f);
    q = __fmaf_rn(q, h, 1.0f / 5040.0f);
    q = __fmaf_rn(q, h, 1.0f / 720.0f);
    q = __fmaf_rn(q, h, 1.0f / 120.0f);
    q = __fmaf_rn(q, h, 1.0f / 24.0f);
    q = __fmul_rn(q, __fmul_rn(square.h, square.h));
    const Two x = two_sum(1.0f, h), y = two_sum(x.h, 0.5f * square.h), z = two_sum(y.h, third.h);
    const float low = __fmaf_rn(r.l, z.h, q) + (((x.l + y.l) + (z.l + third.l)) + 0.5f * square.l);
    return two_sum(z.h, low);
}

// 1 / (a.h + a.l) to 2^-44 of itself.
__device__ __forceinline__ Two two_reciprocal(Two a)
{
    const float h = __frcp_rn(a.h);
    return {h, __fmul_rn(h, __fmaf_rn(-a.l, h, __fmaf_rn(-a.h, h, 1.0f)))};
}

// In units of 2^-40, rounded; sizes below 2^20.
__device__ __forceinline__ long long fixed40(Two a)
{
    constexpr float kOne = 1099511627776.0f;
    return __float2ll_rn(a.h * kOne) + __float2ll_rn(a.l * kOne);
}

// The key of an open expert in units of 2^-40, off by less than 2^-32, where
// |x| (softmax: m - x) is below 80 and |b| below 2^16: the logistic function of x,
// or exp(x - m) times `part`, plus b.
constexpr long long kFixedRoom = 1 << 10;            // keys nearer than this, and sums of two, are left open
constexpr long long kNanKey = -(1ll << 60);          // below every number's
constexpr long long kNoKey = -(1ll << 62);           // below every key and sum of two

__device__ __noinline__ long long fixed_key(float x, float m, Two part, float b, bool softmax)
{
    if (x != x) return kNanKey;
    const Two z = softmax ? two_sum(x, -m) : Two{-x, 0.0f};
    int n;
    Two s = two_exp(z.h, z.l, n);
    s.h = ldexpf(s.h, n);
    s.l = ldexpf(s.l, n);
    if (softmax) {
        const Two p = two_product(s.h, part.h);
        s = {p.h, __fmaf_rn(s.h, part.l, __fmaf_rn(s.l, part.h, p.l))};
    } else {
        const Two d = two_sum(1.0f, s.h);
        s = two_reciprocal(two_sum(d.h, d.l + s.l));
    }
    const Two c = two_sum(s.h, b);
    return fixed40({c.h, c.l + s.l});
}

// The sum of a row's exp(x - m) as its reciprocal, for softmax with a bias
// (without one it divides all alike): added up as integers of 2^-50, to 2^-32 of
// itself, in every lane.
__device__ __noinline__ Two fixed_part(const float *row, int E, float m)
{
    long long all = 0;
    for (int e = threadIdx.x & 31; e < E; e += 32)
        if (row[e] > -INFINITY) all += fixed_key(row[e], m, {1024.0f, 0.0f}, 0.0f, true);
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(kFullMask, all, o);
    constexpr float kOne = 1125899906842624.0f;      // 2^50
    const float h = __ll2float_rn(all);
    const Two part = two_reciprocal({h, __ll2float_rn(all - (long long)h)});
    return {part.h * kOne, part.l * kOne};
}

// A row's reach, for fixed_key: whether all open experts' arguments are in range.
__device__ __noinline__ bool in_range(const float *row, int E, float m, bool softmax, float largest)
{
    float far = largest < 65536.0f ? 0.0f : INFINITY;
    for (int e = threadIdx.x & 31; e < E; e += 32)
        if (row[e] > -INFINITY) far = fmaxf(far, fabsf(softmax ? m - row[e] : row[e]));
    return warp_max(far) < 80.0f;
}

// The groups that stay, `kept` so far, where those in `close` are nearer the
// border than fp32's errors: these are valued again, from the experts that may be
// their best (keys from `from`, each lane's group's), the others keep their side
// of it.  False where that leaves it open too.
__device__ __noinline__ bool careful_groups(const float *keys, const float *row, const float *bias, int E, int group_lanes,
                                            float from, unsigned close, const Rules r, float m, float largest,
                                            bool by_logits, unsigned &kept)
{
    const int lane = threadIdx.x & 31, size = E / r.groups, g = lane / group_lanes;
    __syncwarp();
    if (!in_range(row, E, m, r.softmax, largest)) return false;
    const Two part = r.softmax && r.bias ? fixed_part(row, E, m) : Two{1.0f, 0.0f};
    long long u = kNoKey, v = kNoKey;
    float ux = 0.0f, vx = 0.0f;
    from = fmaxf(from, -FLT_MAX);
    if (g < r.groups && (close >> g & 1))
        for (int e = g * size + lane - g * group_lanes; e < (g + 1) * size; e += group_lanes)
            if (keys[e] >= from) insert(fixed_key(row[e], m, part, bias[e], r.softmax), row[e], u, ux, v, vx);
    __syncwarp();
#pragma unroll 1
    for (int o = group_lanes >> 1; o > 0; o >>= 1) {
        const long long u2 = __shfl_xor_sync(kFullMask, u, o), v2 = __shfl_xor_sync(kFullMask, v, o);
        const float ux2 = __shfl_xor_sync(kFullMask, ux, o), vx2 = __shfl_xor_sync(kFullMask, vx, o);
        insert(u2, ux2, u, ux, v, vx);
        insert(v2, vx2, u, ux, v, vx);
    }
    if (r.group_top == 2 && v > kNoKey) u = v > kNanKey ? u + v : v;
    else vx = 0.0f;
    u = __shfl_sync(kFullMask, u, lane * group_lanes & 31);      // lane g has group g's
    ux = __shfl_sync(kFullMask, ux, lane * group_lanes & 31);
    vx = __shfl_sync(kFullMask, vx, lane * group_lanes & 31);
    int before = 0;
    bool open = false;
#pragma unroll 1
    for (unsigned left = close; left; left &= left - 1) {
        const int h = __ffs(left) - 1;
        const long long o = __shfl_sync(kFullMask, u, h);
        const float ox = __shfl_sync(kFullMask, ux, h), oy = __shfl_sync(kFullMask, vx, h);
        before += o > u || (o == u && h < lane);
        // equal by the same logits or by a NaN, or only nearer than the errors
        open |= (close >> lane & 1) && h != lane && o - u <= kFixedRoom && u - o <= kFixedRoom &&
                !(by_logits && ox == ux && oy == vx) && o != kNanKey;
    }
    const int places = __popc(kept & close);
    kept = (kept & ~close) | __ballot_sync(kFullMask, (close >> lane & 1) && before < places);
    return !__any_sync(kFullMask, open);
}

// Ranks `picks` picks, some nearer than fp32's errors (room): lane k's key and
// expert (-1: none), which becomes its expert by rank.  False where that is open.
__device__ __noinline__ bool careful_picks(int picks, float key, float room, const float *row, const float *bias, int E,
                                           const Rules r, float m, float largest, int &id)
{
    const int lane = threadIdx.x & 31;
    const float x = id >= 0 ? row[id] : -INFINITY, b = id >= 0 ? bias[id] : 0.0f;
    const float next_x = __shfl_down_sync(kFullMask, x, 1), next_b = __shfl_down_sync(kFullMask, b, 1);
    const float next = __shfl_down_sync(kFullMask, key, 1);
    // the same logit and bias twice are in order: the lower index was picked first
    if (!__any_sync(kFullMask, lane < picks - 1 && next > -INFINITY && key - next <= room && (next_x != x || next_b != b)))
        return true;
    if (!in_range(row, E, m, r.softmax, largest)) return false;
    const Two part = r.softmax ? fixed_part(row, E, m) : Two{1.0f, 0.0f};
    const long long v = id >= 0 ? fixed_key(x, m, part, b, r.softmax) : kNoKey;
    __syncwarp();
    int before = 0, source = lane;
    bool open = false;
#pragma unroll 1
    for (int k = 0; k < picks; ++k) {
        const long long o = __shfl_sync(kFullMask, v, k);
        const float ox = __shfl_sync(kFullMask, x, k), ob = __shfl_sync(kFullMask, b, k);
        const int other = __shfl_sync(kFullMask, id, k);
        before += o > v || (o == v && other < id);
        open |= id >= 0 && other >= 0 && o - v <= kFixedRoom && v - o <= kFixedRoom && (ox != x || ob != b);
    }
    if (id < 0) before = lane;                       // these are last already
#pragma unroll 1
    for (int k = 0; k < picks; ++k)
        if (__shfl_sync(kFullMask, before, k) == lane) source = k;
    id = __shfl_sync(kFullMask, id, source);
    return !__any_sync(kFullMask, open);
}

// The choice of one token in 64 bits, by a warp, of the experts that fp32 cannot
// tell apart.  bias: in shared memory, `largest` its largest magnitude; by_logits:
// the picks go by them.  keys, row: E words of shared memory each.  Returns lane
// k's expert, or -1, and its score.
struct Settled {
    int id;
    float score;
};

template <typename L>
__device__ __noinline__ Settled settle(const L *logits, int E, int K, const Rules r, const float *bias, float largest,
                                       bool by_logits, float *keys, float *row)
{
    constexpr double kNan = std::numeric_limits<double>::lowest();
    const int lane = threadIdx.x & 31, size = E / r.groups;
    const bool limited = r.top_groups < r.groups;
    float m = -INFINITY;
    __syncwarp();
    for (int e = lane; e < E; e += 32) {
        row[e] = to_float(logits[e]);
        m = fmaxf(m, row[e]);
    }
    m = warp_max(m);
    float inv = 1.0f, top = -INFINITY;
    double sum = 1.0;                                // softmax's; without a bias it divides all alike
    if (r.softmax) {
        float total = 0.0f;
        for (int e = lane; e < E; e += 32) total += weight_of(row[e], m);
        inv = __fdividef(1.0f, warp_sum(total));
        if (r.bias) {
            sum = 0.0;
            for (int e = lane; e < E; e += 32) sum += row[e] == -INFINITY ? 0.0 : exp((double)row[e] - (double)m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
        }
    }
    const Row scale{m, inv};
    for (int e = lane; e < E; e += 32) {
        const float x = row[e];
        keys[e] = x == -INFINITY ? x : rankable(score_of(x, r, scale) + bias[e]);
        top = fmaxf(top, keys[e]);
    }
    const Room room = room_of(r.softmax ? inv : fminf(fmaxf(warp_max(top) + largest, 0.0f), 1.0f), r.softmax, largest);
    auto exact = [&](int e) {
        const double x = row[e], c = (r.softmax ? exp(x - (double)m) / sum : 1.0 / (1.0 + exp(-x))) + (double)bias[e];
        return c > -INFINITY ? c : kNan;
    };
    __syncwarp();
    unsigned kept = kFullMask;
    if (limited) {
        // As many lanes a group as there are; lane i of them has every such value.
        const int lanes = 32 >> (r.groups == 1 ? 0 : 32 - __clz(r.groups - 1)), g = lane / lanes;
        const int begin = g * size + lane % lanes, end = g < r.groups ? (g + 1) * size : 0;
        float a = -INFINITY, b = -INFINITY;
        for (int e = begin; e < end; e += lanes) insert(keys[e], a, b);
        top_two(a, b, lanes);
        // Every group's value from the experts that may be its best.
        const float from = fmaxf((b > -INFINITY ? b : a) - room.keys, -FLT_MAX);
        double u = -INFINITY, v = -INFINITY;
        for (int e = begin; e < end; e += lanes)
            if (keys[e] >= from) insert(exact(e), u, v);
        top_two(u, v, lanes);
        double value = __shfl_sync(kFullMask, group_value(u, v, r.group_top), lane * lanes & 31);
        if (lane >= r.groups) value = -INFINITY;
        int before = 0;
        for (int h = 0; h < r.groups; ++h) {
            const double o = __shfl_sync(kFullMask, value, h);
            before += o > value || (o == value && h < lane);
        }
        kept = __ballot_sync(kFullMask, lane < r.groups && before < r.top_groups);
    }
    for (int e = lane; e < E; e += 32) {
        const bool in = row[e] > -INFINITY || row[e] != row[e];
        keys[e] = !in || (limited && !(kept >> (e / size) & 1)) ? -INFINITY : by_logits ? rankable(row[e]) : keys[e];
    }
    // The Kth largest key: what is below it by more than the errors is out.
    float least = -FLT_MAX;
    unsigned gone = 0;                               // of this lane's keys, the picks
    for (int k = 0; k < K; ++k) {
        float best = -INFINITY;
        int at = -1;
        for (int i = 0, e = lane; e < E; ++i, e += 32)
            if (!(gone >> i & 1) && keys[e] > best) {
                best = keys[e];
                at = i;
            }
        least = warp_max(best);
        if (!(least > -INFINITY)) break;
        if (lane == __ffs(__ballot_sync(kFullMask, best == least)) - 1) gone |= 1u << at;
    }
    const float from = fmaxf(by_logits ? least : least - room.keys, -FLT_MAX);
    // The candidates in order of experts, 32 of a lane each; each one's place is the
    // number of better ones.  Their list takes the keys' place, from the front: a
    // word is written after all of the words up to it have been read.
    int *const list = reinterpret_cast<int *>(keys);
    int n = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const bool in = e0 + lane < E && keys[e0 + lane] >= from;
        const unsigned all = __ballot_sync(kFullMask, in);
        if (in) list[n + __popc(all & ((1u << lane) - 1))] = e0 + lane;
        n += __popc(all);
        __syncwarp();
    }
    auto exact_key = [&](int e) { return !by_logits ? exact(e) : row[e] == row[e] ? (double)row[e] : kNan; };
    int mine = -1;                                   // what lane k is given, candidate by candidate
    for (int a0 = 0; a0 < n; a0 += 32) {
        const int i = a0 + lane, e = i < n ? list[i] : -1;
        const double v = i < n ? exact_key(e) : 0.0;
        int before = 0;
        for (int b0 = 0; b0 < n; b0 += 32) {
            const double w = b0 == a0 ? v : b0 + lane < n ? exact_key(list[b0 + lane]) : 0.0;
            for (int j = 0; j < min(32, n - b0); ++j) {
                const double o = __shfl_sync(kFullMask, w, j);
                before += o > v || (o == v && b0 + j < i);
            }
        }
        for (int j = 0; j < min(32, n - a0); ++j) {
            const int place = __shfl_sync(kFullMask, before, j), id = __shfl_sync(kFullMask, e, j);
            if (place == lane) mine = id;
        }
    }
    if (lane >= K) mine = -1;
    return {mine, mine >= 0 ? score_of(row[mine], r, scale) : 0.0f};
}

// KT > 0: K is KT, and the picks are unrolled.  single: the grid is one cluster.
template <int NV, int W, int KT, typename L>
__global__ void __launch_bounds__(kWarps * 32, per_sm(NV))
route_grouped_kernel(const L *__restrict__ logits, int T, int E, int any_k, const Rules r,
                     const uint8_t *__restrict__ mask, int32_t *ids, float *__restrict__ weights,
                     uint32_t *__restrict__ part, RouteOut o, bool single)
{
    const int K = KT > 0 ? KT : any_k;
    constexpr int WARPS = kWarps, THREADS = WARPS * 32;
    extern __shared__ float sm[];
    constexpr int PITCH = 32 * NV;                       // a row's words: no lane's values are outside
    constexpr int LIST = list_of(NV);
    float *const sums = sm;                              // [WARPS][PITCH]; until then a warp's keys
    float *const rows = sums + WARPS * PITCH;            // [WARPS][PITCH], a warp's logits
    float *const bias = rows + WARPS * PITCH;            // [PITCH], zeros from E on
    float *const lists = bias + PITCH;                   // [WARPS][32][LIST], a lane's keys sorted, then -inf
    int32_t *const cnt = reinterpret_cast<int32_t *>(lists + WARPS * 32 * LIST);        // [E] and the routed tokens
    uint32_t *const inbox = reinterpret_cast<uint32_t *>(cnt + E + 1);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    for (int e = threadIdx.x; e <= E; e += THREADS) cnt[e] = 0;
    pdl_wait();
    pdl_trigger();
    for (int e = threadIdx.x; e < PITCH; e += THREADS) bias[e] = r.bias && e < E ? r.bias[e] : 0.0f;
    constexpr bool kAhead = NV <= 4;                     // further a lane lacks the registers
    const int stride = gridDim.x * WARPS;
    int t = blockIdx.x * WARPS + warp;
    float ahead[NV];
    uint8_t open = 1;
    const L *next_row = logits + (size_t)t * E;
    const size_t row_step = (size_t)stride * E, id_step = (size_t)stride * K;
    auto fetch = [&](int u) {
        if (u >= T) return;
        load_row<NV, W>(next_row, E, lane, ahead);
        if (mask) open = mask[u];
        next_row += row_step;
    };
    if constexpr (kAhead) fetch(t);
    __syncthreads();

    const int k_lanes = 1 << (32 - __clz(K - 1));        // K, rounded up to a power of two
    const int size = E / r.groups;                       // experts a group
    const bool limited = r.top_groups < r.groups;
    // A group's values are found by group_lanes lanes.  Where a group is that many
    // lanes' own values they need not pass through shared memory; otherwise a
    // lane's first value is number `in_group` of group `my_group`.
    const bool whole = size % NV == 0 && ((size / NV) & (size / NV - 1)) == 0;
    const int group_lanes = whole ? size / NV : 32 >> (r.groups == 1 ? 0 : 32 - __clz(r.groups - 1));
    const int my_group = lane * NV / size, in_group = lane * NV - my_group * size;
    float *const key_row = sums + warp * PITCH, *const x_row = rows + warp * PITCH;
    int routed = 0;                                      // tokens with a first pick (lane 0)
    float acc[NV], largest = 0.0f, low = INFINITY, high = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) acc[j] = 0.0f;
    {
        float b[NV];
        load_own<NV>(bias, lane, b);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (lane * NV + j < E) {
                low = fminf(low, b[j]);
                high = fmaxf(high, b[j]);
            }
        }
    }
    low = -warp_max(-low);
    high = warp_max(high);
    largest = fmaxf(fabsf(low), fabsf(high));
    const bool by_logits = low == high;                  // no bias, or one for all
    bool again = false;                                  // some token's choice is open

    // A token's weights, counts and ids from lane k's expert and its score.
    auto finish = [&](size_t at, int id, float w) {
        if (r.renorm) {
            const float all = lanes_sum(w, k_lanes);
            if (all != 0.0f) w = __fdividef(w, all);
        }
        if (lane < K) {
            ids[at + lane] = id;
            weights[at + lane] = w * r.scale;
        }
        if (id >= 0) atomicAdd(&cnt[id], 1);
        routed += id >= 0;
    };

    // what fp32 cannot tell apart where scores may be up to 1
    const Room most_room = room_of(1.0f, false, largest);
    for (size_t first_id = (size_t)t * K; t < T; t += stride, first_id += id_step) {
        if constexpr (!kAhead) fetch(t);
        float x[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j] = ahead[j];
        const bool masked = !open;
        if constexpr (kAhead) fetch(t + stride);
        if (masked) {
#pragma unroll
            for (int j = 0; j < NV; ++j) x[j] = -INFINITY;
        }
        Row row{0.0f, 0.0f};
        float s[NV], total = 0.0f;
        if (r.softmax) {
            row.m = warp_max(lane_max<NV>(x));
            if (!(row.m > -INFINITY)) row.m = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                s[j] = weight_of(x[j], row.m);
                total += s[j];
            }
            total = warp_sum(total);
            row.inv = total == 0.0f ? 0.0f : __fdividef(1.0f, total);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                s[j] *= row.inv;
                acc[j] += s[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                s[j] = sigmoid_approx(x[j]);
                total += s[j];
            }
            total = warp_sum(total);
            const float inv = total == 0.0f ? 0.0f : __fdividef(1.0f, total);
#pragma unroll
            for (int j = 0; j < NV; ++j) acc[j] += s[j] * inv;
        }
        // key: what the picks go by; -inf where an expert is not open or its group is out
        float key[NV];
        load_own<NV>(bias, lane, key);
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = x[j] == -INFINITY ? x[j] : rankable(s[j] + key[j]);
        __syncwarp();                                    // the last token's are read
        store_own<NV>(key_row, lane, key);
        store_own<NV>(x_row, lane, x);
        Room room = r.softmax ? room_of(row.inv, true, largest) : most_room;
        bool unsure = false;
        if (limited) {
            float a = -INFINITY, c = -INFINITY;
            if (whole) {
                a = key[0];
#pragma unroll
                for (int j = 1; j < NV; ++j) {
                    c = fmaxf(c, fminf(a, key[j]));
                    a = fmaxf(a, key[j]);
                }
            } else {
                __syncwarp();
                const int g = lane / group_lanes;
                if (g < r.groups)
                    for (int i = lane - g * group_lanes; i < size; i += group_lanes) {
                        const float v = key_row[g * size + i];
                        c = fmaxf(c, fminf(a, v));
                        a = fmaxf(a, v);
                    }
                __syncwarp();
            }
            top_two(a, c, group_lanes);
            float value = __shfl_sync(kFullMask, group_value(a, c, r.group_top), lane * group_lanes & 31);
            if (lane >= r.groups) value = -INFINITY;
            // the best groups one by one; lane g has group g's value
            unsigned out = r.groups == 32 ? kFullMask : (1u << r.groups) - 1;
            float rest = value, least = 0.0f;
            for (int k = 0; k < r.top_groups; ++k) {
                least = warp_max(rest);
                const int g = __ffs(__ballot_sync(kFullMask, rest == least) & out) - 1;
                out &= ~(1u << g);
                if (lane == g) rest = -INFINITY;
            }
            unsigned kept = ~out;
            const float most = warp_max(rest);           // above -inf: so are all that stay
            if (most > -INFINITY && least - most <= room.groups) {
                if (!r.softmax) room = room_of(fminf(fmaxf(warp_max(a) + largest, 0.0f), 1.0f), false, largest);
                if (least - most <= room.groups) {
                    const unsigned close = __ballot_sync(kFullMask, value > -INFINITY && value >= least - room.groups &&
                                                                        value <= most + room.groups);
                    unsure = !careful_groups(key_row, x_row, bias, E, group_lanes, (c > -INFINITY ? c : a) - room.keys, close,
                                             r, row.m, largest, by_logits, kept);
                }
            }
            // from shared memory, so that they need no registers past the call above
            load_own<NV>(by_logits ? x_row : key_row, lane, key);
            if (whole) {
                const bool in = kept >> (lane / group_lanes & 31) & 1;
#pragma unroll
                for (int j = 0; j < NV; ++j) key[j] = in ? key[j] : -INFINITY;
            } else {
                int g = my_group, at = in_group;
#pragma unroll
                for (int j = 0; j < NV; ++j, ++at) {
                    if (at == size) {
                        at = 0;
                        ++g;
                    }
                    if (!(kept >> (g & 31) & 1)) key[j] = -INFINITY;
                }
            }
        } else if (by_logits) {
            load_own<NV>(x_row, lane, key);
        }
        if (by_logits) {
#pragma unroll
            for (int j = 0; j < NV; ++j) key[j] = key[j] == -INFINITY ? key[j] : rankable(key[j] + 0.0f);
        }
        __syncwarp();
        store_own<NV>(key_row, lane, key);

        // Pick number `lane`: its key, and the lane that holds it.  Each pick is one
        // maximum over the lanes' best; its owner's next best comes from a sorted list.
        float mine = -INFINITY;
        int from = 0;
        float next[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) next[j] = key[j];
        const float *list = lists + (warp * 32 + lane) * LIST;
        if constexpr (LIST > 0) {
            sort_values<NV>(next);
            store_own<NV>(lists + warp * 32 * LIST + lane * (LIST - NV), lane, next);
            lists[(warp * 32 + lane) * LIST + NV] = -INFINITY;
        }
        float best = LIST > 0 ? next[0] : lane_max<NV>(next);
        auto pick = [&](int k) {
            const float top = warp_max(best);
            const int owner = __ffs(__ballot_sync(kFullMask, best == top)) - 1;
            if (lane == k) {
                mine = top;
                from = owner;
            }
            if constexpr (LIST > 0) {
                if (lane == owner && top > -INFINITY) best = *++list;
            } else if (lane == owner) {
                int at = 0;
#pragma unroll
                for (int j = NV - 1; j >= 0; --j)
                    if (next[j] == top) at = j;
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (j == at) next[j] = -INFINITY;
                best = lane_max<NV>(next);
            }
        };
        if constexpr (KT > 0) {
#pragma unroll
            for (int k = 0; k < KT; ++k) pick(k);
        } else {
            for (int k = 0; k < K; ++k) pick(k);
        }
        // Picks nearer than their errors: then those after them that are as near to the
        // last one are picked too.
        int picks = K;
        bool near = false;
        const float below = __shfl_down_sync(kFullMask, mine, 1);
        if (!by_logits) {
            const float left = warp_max(best), after = lane == K - 1 ? left : below;
            const float gap = lane < K && after > -INFINITY ? mine - after : INFINITY;
            if (__any_sync(kFullMask, gap <= room.keys)) {
                const float last = __shfl_sync(kFullMask, mine, K - 1), top = __shfl_sync(kFullMask, mine, 0);
                if (!r.softmax) room = room_of(fminf(fmaxf(top + largest, 0.0f), 1.0f), false, largest);
                near = __any_sync(kFullMask, gap <= room.keys);
#pragma unroll 1
                for (float next = left; near && next > -INFINITY && last - next <= room.keys; next = warp_max(best)) {
                    if (picks == 32) {
                        unsure = true;               // too many for a warp
                        break;
                    }
                    pick(picks++);
                }
            }
        }
        // A pick's place among its owner's keys, and its logit.  Equal keys are next to
        // one another, and were picked in order.
        unsigned alike = 0;
        if (__any_sync(kFullMask, near || (below == mine && mine > -INFINITY)))
            alike = __match_any_sync(kFullMask, __float_as_int(mine)) & __match_any_sync(kFullMask, from);
        __syncwarp();
        int id = -1;
        float chosen = -INFINITY;
        if (lane < picks && mine > -INFINITY) {
            int before = __popc(alike & ((1u << lane) - 1)), place = 0;
            float owners[NV];
            load_own<NV>(key_row, from, owners);
            if (before == 0) {
#pragma unroll
                for (int j = NV - 1; j >= 0; --j)
                    if (owners[j] == mine) place = j;
            } else {
#pragma unroll 1
                for (place = 0; place < NV - 1; ++place)
                    if (key_row[from * NV + place] == mine && before-- == 0) break;
            }
            id = from * NV + place;
            chosen = x_row[id];
        }
        if (near && !unsure) {
            unsure = !careful_picks(picks, mine, room.keys, x_row, bias, E, r, row.m, largest, id);
            chosen = id >= 0 ? x_row[id] : -INFINITY;
        }
        if (lane >= K) id = -1;
        if (!unsure) {
            finish(first_id, id, id >= 0 ? score_of(chosen, r, row) : 0.0f);
        } else {
            again = true;
            if (lane == 0) ids[first_id] = kOpen;
        }
    }
    if (again) {
        __syncwarp();
        for (t = blockIdx.x * WARPS + warp; t < T; t += stride) {
            if (ids[(size_t)t * K] != kOpen) continue;
            const L *const at = logits + (size_t)t * E;
            const Settled c = settle<L>(at, E, K, r, bias, largest, by_logits, key_row, x_row);
            finish((size_t)t * K, c.id, c.score);
        }
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NV; ++j) key_row[lane * NV + j] = acc[j];
    if (lane == 0) atomicAdd(&cnt[E], routed);
    if (single) route_totals<WARPS, true>(sums, PITCH, cnt, inbox, E, K, part, o);
    else route_totals<WARPS, false>(sums, PITCH, cnt, inbox, E, K, part, o);
}

template <int NV, int W, typename L>
cudaError_t run_grouped(const void *logits, int T, int E, int K, const Rules &r, float coef, const uint8_t *mask,
                        int32_t *ids, float *weights, int32_t *counts, int32_t *routed, float *loss, void *workspace,
                        cudaStream_t s)
{
    constexpr int WARPS = kWarps;
    const size_t smem = route_smem<0>(E) + ((2 * WARPS + 1) * NV + WARPS * list_of(NV)) * 32 * 4;
    const RouteOut o{counts, routed, loss, coef};
    const int single = single_blocks<WARPS>(T, E);
    constexpr int KT = W > 1 ? 8 : 0;                    // as in route.cu
    auto *const kernel = K == KT ? route_grouped_kernel<NV, W, KT, L> : route_grouped_kernel<NV, W, 0, L>;
    if (smem > 40 << 10) {
        const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), smem);
        if (e != cudaSuccess) return e;
    }
    const int blocks = single ? single : route_clusters<WARPS, per_sm(NV)>(T) * kRouteCluster;
    uint32_t *part = static_cast<uint32_t *>(workspace);
    cudaError_t e = launch_pdl_clusters(kernel, dim3(blocks), dim3(WARPS * 32), smem, s,
                                        single ? single : kRouteCluster, static_cast<const L *>(logits),
                                        T, E, K, r, mask, ids, weights, part, o, single > 0);
    if (e != cudaSuccess || single) return e;
    return launch_route_finish(part, blocks / kRouteCluster, E, K, o, s);
}

}  // namespace

size_t route_grouped_workspace_bytes(int T, int E)
{
    return totals_workspace_bytes<kWarps, per_sm(1)>(T, E);  // the most of the kernels' forms
}

cudaError_t launch_route_grouped(const void *logits, int bf16, int T, int E, int K, int softmax, const float *bias,
                                 int groups, int top_groups, int group_top, int renorm, float scale, float coef,
                                 const uint8_t *mask, int32_t *ids, float *weights, int32_t *counts, int32_t *routed,
                                 float *loss, void *workspace, cudaStream_t stream)
{
    const Rules r{bias, softmax, groups, top_groups, group_top, renorm, scale};
#define CALL(NV, W, L)                                                                    \
    run_grouped<NV, W, L>(logits, T, E, K, r, coef, mask, ids, weights, counts, routed, loss, workspace, stream)
    MOE_GROUPED_CASES(CALL, logits);
#undef CALL
}

}  // namespace moe
