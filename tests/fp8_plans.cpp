// Prints the kernels that the FP8 product runs on 256 CUs for each "M K N f32 fused"
// line of its input: "few RT MT" or "tiles TN TM FIRST".
#include <cstdint>
#include <cstdio>

namespace convrot {
struct Fp8Plan {
    int rt, mt, tn, tm;
    int64_t first;
};
Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K, bool f32_out, bool fused, int64_t cus);
} // namespace convrot

int main()
{
    long long M, K, N;
    int f32, fused;
    while (std::scanf("%lld %lld %lld %d %d", &M, &K, &N, &f32, &fused) == 5) {
        const convrot::Fp8Plan p = convrot::fp8_plan(M, N, K, f32, fused, 256);
        if (p.rt)
            std::printf("few %d %d\n", p.rt, p.mt);
        else
            std::printf("tiles %d %d %lld\n", p.tn, p.tm, (long long)p.first);
    }
}
