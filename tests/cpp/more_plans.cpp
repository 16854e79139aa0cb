// How the 8-bit layers and the orthogonalised update run, without a GPU: the C
// entry points of the first with their launches replaced by lines of text, and
// the plans of the second, with a check that its runs cover every stage of every
// tile once and use no slab twice.  Reads lines from stdin:
//   linear|gated M N K op_w unaligned
//   orthogonalize batch M N
// Host code only; addresses are never read.
#include "linear_i8.hip"
#include "orthogonalize.h"

#include <algorithm>
#include <cstdio>
#include <iostream>
#include <map>
#include <set>
#include <sstream>
#include <string>
#include <vector>

namespace dgor {

using namespace newton_schulz;

int device_status() { return GEMM_OK; }
hipError_t launch_i8_ring(const Product &p, const I8Epilogue &, RingTile t, hipStream_t)
{
    printf(" ring %dx%d%s splits=%d", ring_tile_m(t), ring_tile_n(t), p.gated ? " gated" : "", p.splits);
    // every part has stages, and they are all of them
    const int stages = product_stages(p);
    if (p.splits > 1 && !((p.splits - 1) * p.chunk < stages && p.splits * p.chunk >= stages))
        printf(" BAD");
    return hipSuccess;
}
hipError_t launch_i8_rows(const Product &p, const I8Epilogue &, hipStream_t)
{
    printf(" rows blocks=%d%s", (p.M + 15) / 16, p.gated ? " gated" : "");
    return hipSuccess;
}
hipError_t launch_i8_join(const Product &, const I8Epilogue &, hipStream_t)
{
    printf(" join");
    return hipSuccess;
}
hipError_t launch_i8_pack(const I8Pack &r, hipStream_t)
{
    for (int i = 0; i < r.jobs; ++i)
        printf(" copy%s", r.job[i].transpose ? "-turned" : "");
    return hipSuccess;
}

static bool dealt(Which which, int m, int n, int batch, const Way &way)
{
    const long long tiles = batch * tiles_of(which, m, n, way.tile), stages = ceil_div(which == kGram ? n : m, 32);
    const long long rest = tiles - way.whole, all = rest * stages;
    if (way.whole % way.groups != 0 && rest != 0)
        return false;
    std::vector<long long> next(rest, 0);   // stages of each tile that are covered
    std::set<long long> slabs;
    std::map<long long, int> parts;
    for (int w = 0; w < way.groups; ++w) {
        long long unit = (long long)w * way.run;
        const long long last = std::min((long long)(w + 1) * way.run, all);
        while (unit < last) {
            const long long t = unit / stages, begin = t * stages, s0 = unit - begin;
            const long long steps = std::min(last - unit, stages - s0);
            if (next[t] != s0)
                return false;
            next[t] += steps, unit += steps;
            if (steps < stages) {
                if (!slabs.insert(2LL * w + (begin >= (long long)w * way.run ? 1 : 0)).second)
                    return false;
                parts[t]++;
                // the join's arithmetic finds this run
                if (w < begin / way.run || w > (begin + stages - 1) / way.run)
                    return false;
            }
        }
    }
    for (long long t = 0; t < rest; ++t) {
        const int w0 = (int)(t * stages / way.run), w1 = (int)((t * stages + stages - 1) / way.run);
        if (next[t] != stages || (w0 == w1 ? parts.count(t) != 0 : parts[t] != w1 - w0 + 1))
            return false;
    }
    if (!slabs.empty() && (!way.joined || (size_t)(*slabs.rbegin() + 1) * side_of(way.tile) * side_of(way.tile) * 4 > way.slabs))
        return false;
    return true;
}

}  // namespace dgor

int main()
{
    std::string line;
    alignas(16) static char at[16];
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string what;
        in >> what;
        printf("%s:", line.c_str());
        if (what == "orthogonalize") {
            gemm_orthogonalize_params q{};
            in >> q.batch >> q.M >> q.N;
            q.ldg = q.ldo = q.N, q.steps = 2, q.eps = 1e-7, q.scale = 1;
            for (int i = 0; i < 6; ++i)
                q.coefficients[i] = i % 3 == 0 ? 1.5 : i % 3 == 1 ? -0.5 : 0.0;
            dgor::Layout l;
            const int rc = dgor::lay_out(&q, l);
            if (rc != GEMM_OK) {
                printf(" status %d\n", rc);
                continue;
            }
            if (l.small) {
                printf(" small\n");
                continue;
            }
            if (l.strips) {
                printf(" strips");
                // all columns, none of them empty, in what LDS and registers hold
                const int mb = dgor::ceil_div(l.m, 16);
                const size_t groups = (size_t)q.batch * l.strips, part = groups * mb * (mb + 1) / 2 * 1024;
                if (l.width % 32 != 0 || l.mp % 32 != 0 || l.mp < l.m || l.strips * l.width < l.n || l.strips < 1 ||
                    (l.strips - 1) * l.width >= l.n || 4 * l.mp * (l.width + l.mp) > dgor::kSmallBytes ||
                    4 * l.mp * l.width > 1024 * 16 * dgor::kStripUnits ||
                    mb * (l.width / 16) > dgor::kSmallWaves * dgor::kSmallBlocks || mb * (mb + 1) / 2 > 3 * dgor::kSmallWaves ||
                    l.gram < l.x[0] + groups * 4 * l.mp * l.width || l.poly < l.gram + part || l.bytes < l.poly + part)
                    printf(" BAD");
                printf("\n");
                continue;
            }
            const char *names[] = {"gram", "polynomial", "update"};
            for (int i = 0; i < 3; ++i) {
                const dgor::Way &w = l.way[i];
                printf(" %s tile=%d %s%s", names[i], dgor::side_of(w.tile), w.whole ? "whole" : "", w.joined ? "+runs" : "");
                if (!dgor::dealt((dgor::Which)i, l.m, l.n, q.batch, w))
                    printf(" BAD");
            }
            printf("\n");
            continue;
        }
        int M, N, K, op, off;
        in >> M >> N >> K >> op >> off;
        const int8_t *x = (const int8_t *)at;
        const float *f = (const float *)at;
        size_t need = 0;
        int rc;
        void *ws = (void *)0x1000;
        if (what == "linear") {
            gemm_linear_i8_params q{M, N, K, op, K, op ? K : N, N, N, 1, off};
            rc = gemm_linear_i8_workspace(&q, &need);
            if (rc == GEMM_OK)
                rc = gemm_linear_i8_f32(&q, x, f, x, f, nullptr, nullptr, (float *)at, ws, need, nullptr);
        } else {
            gemm_gated_i8_params q{M, N, K, op, K, op ? K : N, N, 1, off};
            rc = gemm_gated_i8_workspace(&q, &need);
            if (rc == GEMM_OK)
                rc = gemm_gated_i8_f32(&q, x, f, x, f, x, f, (float *)at, ws, need, nullptr);
        }
        printf(" status %d\n", rc);
    }
    return 0;
}
