// tern_route.hip -- the experts that tokens take, and their weights, from a
// router's logits.
//
// Mathematics, for a token with logits l over E experts:
//   s = softmax of l over the experts, or sigmoid of each l
//   c = s + bias, what is chosen by; without a bias the order of the logits, which
//       is the same where s does not run out of bits
//   with G groups of E / G consecutive experts, only those of the `keep` groups
//       with the largest sums of their `best` (1 or 2) largest c are open
//   S = the top_k open experts by c, w = s, divided by their sum over S if
//       renormalised, times a factor
// Equal values go to the lowest index, for groups as for experts.  An expert whose
// logit (or c) is -inf is never taken; a NaN counts as the largest.
//
// A choice hangs on the last bit of c, so s and c are formed in 64 bits where the
// order of the logits does not do, and the weights of the chosen experts, one a
// lane, everywhere.
//
// Work layout.  A wave takes a token, lane i the experts i, 64 + i, ...; the chosen
// ones are found one after another, a maximum over the wave each.
//
// Bound: latency, the launch and a chain of maxima over the wave: 1 token of 256
// experts, sigmoid with a bias, 8 groups, 8 chosen 7.4 us; 8192 tokens of 128 experts,
// softmax, 8 chosen 8.4 us, of which reading 2 MB of logits takes 2.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "tern_route.h"
#include "tern_route_device.h"

namespace tern {

namespace {

// Key: 32 bits, the logits' order, or 64, that of c.  E <= 64 R.
template <typename Key, int R>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
    constexpr bool WIDE = sizeof(Key) == 8;
    extern __shared__ uint64_t lds64[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int E = a.E, per = E / a.groups;
    Key *keys = reinterpret_cast<Key *>(lds64) + wave * E;   // groups only
    const float ninf = -__builtin_inff();
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.T; t += (int64_t)gridDim.x * 4) {
        float l[R];
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int e = 64 * i + lane;
            l[i] = e < E ? load_logit(a.logits, a.l_dtype, t * E + e) : ninf;
            most = max(most, order_key(l[i]));
        }
        // the largest logit; no score of a softmax is a number where that is infinite
        const float largest = key_value(wave_max(most));
        const double top = a.sigmoid ? 0.0 : (double)(largest == -ninf ? __builtin_nanf("") : largest);
        // what a logit's score is before the division by `total`
        auto score = [&](float v) __attribute__((always_inline)) {
            return a.sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : v == ninf ? 0.0 : exp((double)v - top);
        };
        double total = 1.0;   // of all scores, where they are needed as they are
        if (!a.sigmoid && (WIDE || !a.renormalize)) {
            double part = 0.0;
#pragma unroll
            for (int i = 0; i < R; ++i) part += score(l[i]);
            total = wave_sum(part);
        }
        Key key[R];   // 0: not open
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int e = 64 * i + lane;
            if constexpr (WIDE) {
                const double c = score(l[i]) / total + (a.bias != nullptr && e < E ? (double)a.bias[e] : 0.0);
                key[i] = l[i] == ninf || c == (double)ninf ? 0 : order_key(c);
            } else {
                key[i] = l[i] == ninf ? 0 : order_key(l[i]);
            }
        }
        if (a.groups > 1) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (64 * i + lane < E) keys[64 * i + lane] = key[i];
            wave_order();
            // `each` lanes for a group, which then hold its two largest keys
            int each = 64;
            while (each * a.groups > 64) each >>= 1;
            const int g = lane / each, at = lane % each;
            Key b1 = 0, b2 = 0;
            if (g < a.groups)
                for (int j = at; j < per; j += each) {
                    const Key k = keys[g * per + j];
                    b2 = max(b2, min(b1, k)), b1 = max(b1, k);
                }
            for (int d = 1; d < each; d <<= 1) {
                const Key o1 = (Key)__shfl_xor((unsigned long long)b1, d), o2 = (Key)__shfl_xor((unsigned long long)b2, d);
                b2 = max(max(b2, o2), min(b1, o1)), b1 = max(b1, o1);
            }
            if constexpr (WIDE)
                if (a.best == 2 && b2 != 0) b1 = order_key(key_value(b1) + key_value(b2));
            int before = 0;   // groups that come first
            for (int o = 0; o < a.groups; ++o) {
                const Key k = (Key)__shfl((unsigned long long)b1, o * each);
                before += k > b1 || (k == b1 && o < g);
            }
            const uint64_t kept = __ballot(g < a.groups && at == 0 && before < a.keep);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int e = min(64 * i + lane, E - 1);
                if (!(kept >> (e / per * each) & 1)) key[i] = 0;
                // groups go by sums of scores, experts without a bias by their logits
                if constexpr (WIDE)
                    if (a.bias == nullptr && key[i] != 0) key[i] = order_key((double)l[i]);
            }
            wave_order();
        }
        int id = -1;
        float mine = 0.f;   // the logit of the lane's choice
        for (int j = 0; j < a.top_k; ++j) {
            Key m = key[0];
#pragma unroll
            for (int i = 1; i < R; ++i) m = max(m, key[i]);
            m = wave_max(m);
            if (m == 0) break;
            int e = -1;   // the lowest index that holds it
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const uint64_t hit = __ballot(key[i] == m);
                if (e < 0 && hit != 0) {
                    const int at = __ffsll((unsigned long long)hit) - 1;
                    e = 64 * i + at;
                    v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, l[i]), at));
                    if (lane == at) key[i] = 0;
                }
            }
            if (lane == j) id = e, mine = v;
        }
        double w = id >= 0 ? score(mine) : 0.0;
        if (a.renormalize) total = wave_sum(w);
        // none for a place without an expert, whatever the factor and the others' scores are
        w = total == 0.0 || id < 0 ? 0.0 : w / total * (double)a.scale;
        if (lane < a.top_k) {
            a.ids[t * a.top_k + lane] = id;
            a.weights[t * a.top_k + lane] = (float)w;
        }
    }
}

template <typename Key, int R>
hipError_t launch_t(const RouteArgs &a) {
    const unsigned grid = (unsigned)std::min<int64_t>((a.T + 3) / 4, 2048);
    const size_t lds = a.groups > 1 ? (size_t)4 * a.E * sizeof(Key) : 0;
    hipLaunchKernelGGL((route_kernel<Key, R>), dim3(grid), dim3(256), lds, a.stream, a);
    return hipGetLastError();
}

template <typename Key>
hipError_t launch_k(const RouteArgs &a) {
    if (a.E <= 64) return launch_t<Key, 1>(a);
    if (a.E <= 128) return launch_t<Key, 2>(a);
    if (a.E <= 256) return launch_t<Key, 4>(a);
    if (a.E <= 512) return launch_t<Key, 8>(a);
    return launch_t<Key, 16>(a);
}

}  // namespace

hipError_t launch_route(const RouteArgs &a) {
    return a.bias != nullptr || (a.groups > 1 && a.best == 2) ? launch_k<uint64_t>(a) : launch_k<uint32_t>(a);
}

}  // namespace tern
