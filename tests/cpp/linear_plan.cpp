// The dense layers' C entry points with their launches replaced by lines of
// text: which kernel, tile, layout and split each product of a call takes, and
// how many threads a launch has.  Reads calls from stdin, one a line:
//   name format shift-of-each-pointer... : parameters...
// where a shift is the pointer's distance in bytes from a 256-byte boundary, or
// -1 for NULL.  Host code only; addresses are never read.
#include "linear.hip"

#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

namespace dgor {

static const char *layout(const Product &p)
{
    return p.gated ? (p.trans_b ? "gated NxK" : "gated KxN") : p.trans_a ? "KxM" : p.trans_b ? "NxK" : "KxN";
}
static void product(const char *kernel, const Product &p, int tm, int tn, long long threads)
{
    const long long tiles = (long long)((p.M + tm - 1) / tm) * ((p.N + (p.gated ? tn / 2 : tn) - 1) / (p.gated ? tn / 2 : tn));
    double us = 0;   // what a ring was chosen for, its join included; printed in tenths
    for (const RingCost &c : kRings)
        if (threads == 256 && ring_tile_m(c.tile) == tm && ring_tile_n(c.tile) == tn)
            us = microseconds(p, c, tiles * p.nbatch, p.splits > 1 ? p.splits : 1);
    printf("%s tile=%dx%d layout=%s M=%d N=%d K=%d segments=%d terms=%d batches=%d splits=%d chunk=%d stages=%d "
           "threads=%lld estimate=%d\n",
           kernel, tm, tn, layout(p), p.M, p.N, p.K, p.nseg, p.terms, p.nbatch, p.splits > 1 ? p.splits : 1, p.chunk,
           product_stages(p), tiles * p.nbatch * threads, (int)(10 * us + 0.5));
}

int device_status() { return GEMM_OK; }
hipError_t launch_tile(const Product &p, hipStream_t)
{
    product("tile", p, kTile, kTile, 256);
    return hipSuccess;
}
hipError_t launch_linear_ring(const Product &p, RingTile t, hipStream_t)
{
    product("ring", p, ring_tile_m(t), ring_tile_n(t), 256);
    return hipSuccess;
}
hipError_t launch_linear_ring_pair(const Product &w, const Product &x, RingTile t, hipStream_t)
{
    product("pair", w, ring_tile_m(t), ring_tile_n(t), 256);
    product("pair", x, ring_tile_m(t), ring_tile_n(t), 256);
    return hipSuccess;
}
hipError_t launch_linear_skinny(const Product &p, hipStream_t)
{
    const int strip = skinny_strip(p, p.splits > 1) * (p.gated ? 2 : 1);   // product() halves a gated tile
    product("rows", p, kSkinnyRows, strip, 512);
    return hipSuccess;
}
hipError_t launch_repack(const Repack &r, hipStream_t)
{
    if (r.jobs)
        printf("copies jobs=%d opened=%d\n", r.jobs, r.job[0].lo != nullptr);
    return hipSuccess;
}
hipError_t launch_join(const Product &p, hipStream_t)
{
    printf("join batches=%d threads=%lld\n", p.nbatch, (long long)p.M * ((p.N + 7) / 8));
    return hipSuccess;
}
hipError_t launch_act_grad(int M, int N, const uint16_t *, int, const uint16_t *, int, uint16_t *dz, uint16_t *lo, int, int,
                           float *, uint16_t *, const Repack &r, bool, hipStream_t)
{
    printf("act_grad terms=%d copies=%d threads=%lld\n", dz ? (lo ? 2 : 1) : 0, r.jobs, 256LL * grad_groups(M, N));
    return hipSuccess;
}
hipError_t launch_sum_blocks(int blocks, int, const float *, uint16_t *, bool, hipStream_t)
{
    printf("sum_blocks blocks=%d\n", blocks);
    return hipSuccess;
}
hipError_t launch_gate_grad(int M, int F, const uint16_t *, int, const uint16_t *, const uint16_t *, int,
                            const GateGrads &d, int, int, const Repack &r, bool, hipStream_t)
{
    printf("gate_grad terms=%d copies=%d threads=%lld\n", d.g[1] ? 2 : 1, r.jobs, 256LL * gate_groups(M, F));
    return hipSuccess;
}

}  // namespace dgor

template <class Params>
static Params read(std::istream &in)
{
    Params p{};
    int *at = reinterpret_cast<int *>(&p);
    for (size_t i = 0; i < sizeof(Params) / sizeof(int); ++i)
        in >> at[i];
    return p;
}

int main()
{
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string name, format, word;
        in >> name >> format;
        std::vector<uint16_t *> v;
        while (in >> word && word != ":") {
            const long long shift = std::stoll(word);
            // 2^44 apart: no operand reaches the next
            v.push_back(shift < 0 ? nullptr : (uint16_t *)(((uintptr_t)(v.size() + 1) << 44) + shift));
        }
        void *const ws = (void *)(1ull << 60);
        const size_t all = ~(size_t)0 >> 8;
        const bool b = format == "bf16";
        size_t bytes = 0;
        int rc = -100;
        if (name == "linear") {
            const auto p = read<gemm_linear_params>(in);
            gemm_linear_workspace(&p, &bytes);
            rc = run_linear(b, &p, v[0], v[1], v[2], v[3], v[4], v[5], ws, all, nullptr);
        } else if (name == "linear_backward") {
            const auto p = read<gemm_linear_backward_params>(in);
            gemm_linear_backward_workspace(&p, &bytes);
            rc = run_linear_backward(b, &p, v[0], v[1], v[2], v[3], v[4], v[5], v[6], ws, all, nullptr);
        } else if (name == "gated") {
            const auto p = read<gemm_gated_params>(in);
            gemm_gated_workspace(&p, &bytes);
            rc = run_gated(b, &p, v[0], v[1], v[2], v[3], v[4], v[5], ws, all, nullptr);
        } else if (name == "gated_backward") {
            const auto p = read<gemm_gated_backward_params>(in);
            gemm_gated_backward_workspace(&p, &bytes);
            rc = run_gated_backward(b, &p, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], ws, all, nullptr);
        }
        printf("status=%d workspace=%zu\n", rc, bytes);
    }
    return 0;
}
