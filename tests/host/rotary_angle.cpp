// The kernel's angles, on the host: reads lines "i <position> <frequency>" or "f <position>
// <frequency>" (hexadecimal floats), writes the phase, in turns times 2^64.
#include <cinttypes>
#include <cstdio>

#include "rotary_angle.cuh"

int main()
{
    using namespace gbssim;
    char kind, x[64], f[64];
    while (std::scanf(" %c %63s %63s", &kind, x, f) == 3) {
        double rate = 0, at = 0;
        std::sscanf(f, "%la", &rate);
        const turns64 fraction = turn_fraction(rate);
        if (kind == 'i') {
            long long whole = 0;
            std::sscanf(x, "%lld", &whole);
            std::printf("%llu\n", turn_phase(whole, fraction));
        } else {
            std::sscanf(x, "%la", &at);
            std::printf("%llu\n", turn_phase(float(at), fraction, whole_turns(rate), rate < 0));
        }
    }
}
