// What the orthogonalised update's plan makes of its coefficients, without a GPU.
// Reads lines `scale steps a b c ...` from stdin; writes the status and, of each
// step, the exponents of X, A and P.  Host code only.
#include "orthogonalize.h"

#include <cstdio>
#include <cstdlib>
#include <iostream>
#include <sstream>
#include <string>

int main()
{
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        gemm_orthogonalize_params q{};
        q.batch = 1, q.M = q.N = q.ldg = q.ldo = 200, q.eps = 1e-7;
        std::string number;
        in >> number >> q.steps;
        q.scale = std::strtod(number.c_str(), nullptr);
        for (int i = 0; i < 3 * q.steps; ++i) {
            in >> number;
            q.coefficients[i] = std::strtod(number.c_str(), nullptr);
        }
        dgor::newton_schulz::Layout l;
        const int rc = dgor::newton_schulz::lay_out(&q, l);
        printf("%d", rc);
        for (int i = 0; rc == GEMM_OK && i < q.steps; ++i)
            printf(" %d %d %d", l.step[i].x, l.step[i].gram, l.step[i].poly);
        printf("\n");
    }
    return 0;
}
